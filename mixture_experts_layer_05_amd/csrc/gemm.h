// Matrix products c[m, n] = sum_k a(m, k) b(n, k) whose operands lie in memory either
// with a row's contraction elements side by side (k-contiguous, as x and the weights of
// x W^T) or with the rows' elements of one k side by side (k-strided, as both operands of
// a weight's gradient dy^T x).  What becomes of the sums is the epilogue's, a functor.
//
// Sums run in float32 (8-bit integers: exactly, in int32) over the whole contraction.
#pragma once

#include <algorithm>
#include <type_traits>

#include "dense.h"
#include "dma.h"

namespace moe {
namespace {

enum class El { F32, BF16, I8 };
template <El E>
struct ElInfo {
  static constexpr int kSize = E == El::F32 ? 4 : E == El::BF16 ? 2 : 1;
  static constexpr int kPiece = 16 / kSize;       // elements of 16 bytes
  static constexpr int kStage = 128 / kSize;      // contraction elements of a stage
};

// One operand.  k-contiguous: row r starts ld elements after row r - 1; k-strided: the
// elements of k start ld elements after those of k - 1.
//   q != null, k-contiguous: two matrices whose rows take turns in a tile;
//   q != null, k-strided: k in [0, half) is p's, k in [half, 2 half) q's; of either
//   half the first `live` exist, the others are zeros.
struct Operand {
  const void *p, *q;
  int64_t ld;
  int half, live;
};

// M x N results (a pair of results for each with a k-contiguous pair in b) over K.
struct Product {
  Operand a, b;
  int M, N, K;
};

// 16 bytes of a row that holds `left` more elements, zeros past its end.
template <El E, bool ANY>
__device__ __forceinline__ uint4 piece_of(const uint8_t* p, int left) {
  if constexpr (E == El::F32) {
    if constexpr (ANY) {
      if (left >= 4) {
        const f32x4_any v = *reinterpret_cast<const f32x4_any*>(p);
        return uint4{__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
      }
    }
    return ld_f32x4(p, left, !ANY);
  } else if constexpr (E == El::BF16) {
    return ld8_bf16<ANY>(reinterpret_cast<const uint16_t*>(p), left);
  } else {
    if (left >= 16) {
      if constexpr (!ANY) return ld16(p);
      typedef uint32_t u32x4_b __attribute__((ext_vector_type(4), aligned(1)));
      const u32x4_b v = *reinterpret_cast<const u32x4_b*>(p);
      return uint4{v.x, v.y, v.z, v.w};
    }
    uint32_t v[4] = {0, 0, 0, 0};
    if constexpr (ANY) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (k < left) v[k >> 2] |= static_cast<uint32_t>(p[k]) << (8 * (k & 3));
    }
    return uint4{v[0], v[1], v[2], v[3]};
  }
}

typedef int i32x4v __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
template <El E>
using Acc = std::conditional_t<E == El::I8, i32x16, f32x16>;

// 32 x 32 sums over the 2 x 16 bytes of two lane halves.
template <El E>
__device__ __forceinline__ Acc<E> mfma32(const uint4& a, const uint4& b, Acc<E> c) {
  if constexpr (E == El::F32) {
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  } else if constexpr (E == El::BF16) {
    return mfma_bf16_32x32x16(a, b, c);
  } else {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4v, a), __builtin_bit_cast(i32x4v, b), c, 0, 0, 0);
  }
}

// A sum as it is staged (by value: a bit cast of a vector's element takes element 0).
__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(int v) { return __int_as_float(v); }
// Staged sums added, and as an epilogue takes them: those of 8-bit products stay integers
// until they are whole, so that however a product is split its sums are exact.
template <El E>
__device__ __forceinline__ float add_sums(float a, float b) {
  if constexpr (E == El::I8) return __int_as_float(__float_as_int(a) + __float_as_int(b));
  else return a + b;
}
template <El E>
__device__ __forceinline__ f32x4 whole_sums(const f32x4& s) {
  if constexpr (E != El::I8) return s;
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = s[e];
    r[e] = static_cast<float>(__float_as_int(v));
  }
  return r;
}

// Two reads of 64 bits, each of which turns a 4 (k) x 16 block of a k-strided operand
// between the 16 lanes that address it: lane i gets column i's four elements.
__device__ __forceinline__ uint2 lds_turned(const uint8_t* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)(p)));
}

// ---------------------------------------------------------------- results
//
// An epilogue takes four neighbouring columns of a row at a time:
//   Cols cols(n)                  what it needs of columns n to n + 3
//   Ahead ahead(m, n)             what it reads of row m there, as loaded
//   put(m, n, s, u, cols, ahead)  the results of the sums s (and u, of a pair)
//   kAhead                        the rows of a batch in aligned tiles, by its registers
//   bytes()                       what it reads and writes of a result (the host asks)
// Rows past the end are left out by its caller.

// The rows behind D rows of staged sums, from row R on, and what is read for them.
template <class Epi, int D>
struct Batch {
  int m[D];
  typename Epi::Ahead a[D];
  template <class RowOf>
  __device__ __forceinline__ void load(const Epi& epi, int M, int n, int R, int step, RowOf row_of) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      m[d] = row_of(R + d * step);
      if (m[d] < M) a[d] = epi.ahead(m[d], n);
    }
  }
};

// ROWS x BN sums in LDS, rows `stride` floats apart, to the epilogue or to part p's sums:
// row_of(R) is the row of the product behind row R, and `from` the first of these rows.
// Whole row segments, four columns to a thread.  A PAIR's columns take turns, TURN of the
// first product and TURN of the second.  A part's sums go to part_of(R), those of the second
// product `second` floats on; null leaves a row out.  Sums of 8-bit products are staged as
// the integers they are.  What the epilogue reads for D rows is in flight while D others
// are finished: `now` holds what it reads for the first, and then for the D rows behind the
// last (if `more`).
template <El E, bool PAIR, int TURN, int BN, int ROWS, int THREADS, int D, class Epi, class RowOf, class PartOf>
__device__ __forceinline__ void results_out(const Product& g, const Epi& epi, const typename Epi::Cols& cols, Batch<Epi, D>& now,
                                            const float* stg, int stride, int n, int tid, int from, bool more, RowOf row_of,
                                            bool cut, PartOf part_of, size_t second) {
  constexpr int kLanes = (PAIR ? BN / 2 : BN) / 4, kIter = ROWS * kLanes / THREADS, kStep = THREADS / kLanes;
  static_assert(THREADS % kLanes == 0 && kIter % D == 0, "a thread keeps its columns");
  if (n >= g.N) return;
  const int c = 4 * (tid % kLanes), sc = PAIR ? c / TURN * 2 * TURN + c % TURN : c;
#pragma unroll 1
  for (int k = 0; k < kIter; k += D) {
    const int R = tid / kLanes + k * kStep;
    f32x4 s[D], u[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      s[d] = *reinterpret_cast<const f32x4*>(stg + (R + d * kStep) * stride + sc);
      if constexpr (PAIR) u[d] = *reinterpret_cast<const f32x4*>(stg + (R + d * kStep) * stride + sc + TURN);
    }
    if (cut) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        float* q = part_of(from + R + d * kStep);
        if (!q) continue;
        *reinterpret_cast<f32x4*>(q) = s[d];
        if constexpr (PAIR) *reinterpret_cast<f32x4*>(q + second) = u[d];
      }
      continue;
    }
    Batch<Epi, D> next;
    if (more || k + D < kIter) next.load(epi, g.M, n, from + R + D * kStep, kStep, row_of);
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (now.m[d] < g.M) epi.put(now.m[d], n, whole_sums<E>(s[d]), u[d], cols, now.a[d]);
    now = next;
  }
}

// The parts' sums added in order.
constexpr int kSumAhead = 4;
template <El E, bool PAIR, class Epi>
__global__ void __launch_bounds__(256) product_sum_kernel(Product g, Epi epi, int parts, const float* part) {
  const int quads = static_cast<int>(part_stride(g.N) / 4);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t plane = static_cast<int64_t>(g.M) * quads;
  if (i >= plane) return;
  const f32x4* v = reinterpret_cast<const f32x4*>(part) + i;
  f32x4 s = {0.f, 0.f, 0.f, 0.f}, u = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; p += kSumAhead) {
    f32x4 b[kSumAhead], c[kSumAhead];
#pragma unroll
    for (int k = 0; k < kSumAhead; ++k)
      if (p + k < parts) {
        b[k] = v[plane * (PAIR ? 2 * (p + k) : p + k)];
        if constexpr (PAIR) c[k] = v[plane * (2 * (p + k) + 1)];
      }
#pragma unroll
    for (int k = 0; k < kSumAhead; ++k)
      if (p + k < parts)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[e] = add_sums<E>(s[e], b[k][e]);
          if constexpr (PAIR) u[e] += c[k][e];
        }
  }
  const int m = static_cast<int>(i / quads), n = 4 * static_cast<int>(i - static_cast<int64_t>(m) * quads);
  epi.put(m, n, whole_sums<E>(s), u, epi.cols(n), epi.ahead(m, n));
}

// ---------------------------------------------------------------- tiles of any alignment
//
// BM x BN sums per workgroup of 2 x 2 waves, from 32x32 MFMAs: float32, and what does not
// lie in whole 16-byte pieces.  A stage is 128 bytes of contraction (64 bf16, 32 f32, 128
// int8), double-buffered in LDS; its loads go to registers two to four stages ahead, which
// takes any alignment and fills ends with zeros.  A
// k-contiguous operand's rows lie unpadded in LDS, their 16-byte pieces permuted by
// (row / 2) mod 8; a k-strided one's rows are the k, padded so that the four k that a
// fragment read takes lie in different quarters of the banks.
//
// Bound by the f32 matrix rate where tiles are many, below that by a stage's latency: a
// barrier, the LDS's writes and reads and 16 MFMAs of 64 cycles take about 1 us where the
// MFMAs alone are 0.45.  333 x 515 x 1023 in f32 with odd rows takes 11 to 19 us a product,
// six of them and three sums 99 us in a training step (135 in 64 x 128 and 128 x 128 tiles with
// two stages ahead, 118 in 64 x 64).  Five LDS slots, or the next quarter's fragments read
// ahead, change nothing there.
template <El E, bool KC, int R>
struct TileSide {
  using I = ElInfo<E>;
  static_assert(KC || E != El::I8, "8-bit operands are k-contiguous");
  static constexpr int kRow = KC ? 128 : R * I::kSize + (E == El::F32 ? 32 : 64);
  static constexpr int kBytes = KC ? R * 128 : I::kStage * kRow;
  static constexpr int kPer = KC ? 8 : R / I::kPiece;           // pieces of a row
  static constexpr int kStep = 256 / kPer;                      // rows between a thread's pieces
  static constexpr int kN = (KC ? R : I::kStage) / kStep;       // pieces of a thread
};

template <El E, bool KA, bool KB, bool PAIR, bool ANY, int BM, int BN, class Epi>
__global__ void __launch_bounds__(256, 2) product_tile_kernel(Product g, Epi epi, int parts, float* part) {
  using I = ElInfo<E>;
  using SA = TileSide<E, KA, BM>;
  using SB = TileSide<E, KB, BN>;
  constexpr int NI = BM / 64, NJ = BN / 64, kCols = PAIR && KB ? BN / 2 : BN;
  constexpr bool kPair = PAIR && KB;
  // Of a pair a wave's 32 or 64 columns are half the first product's and half the second's.
  constexpr int kStride = BN + 8, kTurn = BN / 4 < 32 ? BN / 4 : 32;
  constexpr int kBytes = 2 * (SA::kBytes + SB::kBytes) > 64 * kStride * 4 ? 2 * (SA::kBytes + SB::kBytes) : 64 * kStride * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kBytes];
  constexpr int kStageBytes = SA::kBytes + SB::kBytes;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hi = lane >> 5;
  const int mt = static_cast<int>(ceil_div(g.M, BM)), nt = static_cast<int>(ceil_div(g.N, kCols));
  const int item = xcd_tile(blockIdx.x, mt * nt * parts);
  if (item < 0) return;
  const int p = item % parts, m0 = (item / parts) % mt * BM, n0 = (item / parts) / mt * kCols;
  const int stages = static_cast<int>(ceil_div(g.K, I::kStage));
  const int s0 = static_cast<int>(static_cast<int64_t>(p) * stages / parts), s1 = static_cast<int>(static_cast<int64_t>(p + 1) * stages / parts);

  // k-contiguous: thread t loads piece t % 8 of rows t / 8 + 32 q, rows past the end
  // repeat the last.  k-strided: piece t % kPer of k t / kPer + kStep q.
  const uint8_t* ap[SA::kN];
  const uint8_t* bp[SB::kN];
  const int arow = tid / SA::kPer, apiece = tid % SA::kPer, brow = tid / SB::kPer, bpiece = tid % SB::kPer;
  // k-strided: columns that the thread's piece holds, none or less where it is past the end.
  const int aleft = g.M - m0 - apiece * I::kPiece, bleft = g.N - n0 - bpiece * I::kPiece;
  const int apast = aleft > 0 ? 0 : static_cast<int>(ceil_div(1 - aleft, I::kPiece)), bpast = bleft > 0 ? 0 : static_cast<int>(ceil_div(1 - bleft, I::kPiece));
#pragma unroll
  for (int q = 0; q < SA::kN; ++q) {
    if constexpr (KA)
      ap[q] = static_cast<const uint8_t*>(g.a.p) + (static_cast<size_t>(min(m0 + arow + SA::kStep * q, g.M - 1)) * g.a.ld) * I::kSize + 16 * apiece;
    else
      ap[q] = static_cast<const uint8_t*>(g.a.p) + (static_cast<size_t>(arow + SA::kStep * q) * g.a.ld + m0) * I::kSize + 16 * (apiece - apast);
  }
#pragma unroll
  for (int q = 0; q < SB::kN; ++q) {
    const int r = brow + SB::kStep * q;
    if constexpr (kPair) {
      const void* w = (r & kTurn) ? g.b.q : g.b.p;
      bp[q] = static_cast<const uint8_t*>(w) + (static_cast<size_t>(min(n0 + r / (2 * kTurn) * kTurn + r % kTurn, g.N - 1)) * g.b.ld) * I::kSize + 16 * bpiece;
    } else if constexpr (KB) {
      bp[q] = static_cast<const uint8_t*>(g.b.p) + (static_cast<size_t>(min(n0 + r, g.N - 1)) * g.b.ld) * I::kSize + 16 * bpiece;
    } else {
      bp[q] = static_cast<const uint8_t*>(g.b.p) + (static_cast<size_t>(r) * g.b.ld + n0) * I::kSize + 16 * (bpiece - bpast);
    }
  }
  struct Regs {
    uint4 a[SA::kN], b[SB::kN];
  };
  // The stages [0, full), of a k-strided pair also [up, up + full), are loaded without a
  // condition, which keeps several on their way: no k of theirs is past an end.  A piece of
  // a k-strided row may reach past the row's end, into the next row at most, so the last
  // row, and rows shorter than a piece, are no such stage's.  The sums of columns past the
  // end are not stored.
  constexpr bool kStrided = !KA || !KB;
  const int rows = PAIR && !KB ? g.b.live : g.K;
  int full = ANY && kStrided ? (rows - 1) / I::kStage : rows / I::kStage;
  if (ANY && ((!KA && g.a.ld < I::kPiece) || (!KB && g.b.ld < I::kPiece))) full = 0;
  const int up = PAIR && !KB ? g.b.half / I::kStage : stages;
  auto fast = [](const uint8_t* p) __attribute__((always_inline)) {
    typedef uint32_t u32x4_el __attribute__((ext_vector_type(4), aligned(1)));
    if constexpr (!ANY) return ld16(p);
    const u32x4_el v = *reinterpret_cast<const u32x4_el*>(p);
    return uint4{v.x, v.y, v.z, v.w};
  };
  auto load_full = [&](Regs& R, int st) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < SA::kN; ++q)
      R.a[q] = fast(ap[q] + (KA ? static_cast<size_t>(st) * 128 : static_cast<size_t>(st) * I::kStage * g.a.ld * I::kSize));
    // (Of a pair the second matrix instead of the first, from its own first row.)
    const ptrdiff_t over = PAIR && !KB && st >= up ? static_cast<const uint8_t*>(g.b.q) - static_cast<const uint8_t*>(g.b.p) : 0;
    const int row = PAIR && !KB && st >= up ? st - up : st;
#pragma unroll
    for (int q = 0; q < SB::kN; ++q)
      R.b[q] = fast(bp[q] + (KB ? static_cast<size_t>(st) * 128 : static_cast<size_t>(row) * I::kStage * g.b.ld * I::kSize) + over);
  };
  auto load_part = [&](Regs& R, int st) __attribute__((always_inline)) {
    const int k0 = st * I::kStage;
#pragma unroll
    for (int q = 0; q < SA::kN; ++q) {
      if constexpr (KA) {
        R.a[q] = piece_of<E, ANY>(ap[q] + static_cast<size_t>(st) * 128, g.K - k0 - apiece * I::kPiece);
      } else {
        const bool ok = k0 + arow + SA::kStep * q < g.K;
        R.a[q] = piece_of<E, ANY>(ap[q] + static_cast<size_t>(k0) * g.a.ld * I::kSize, ok ? aleft : 0);
      }
    }
#pragma unroll
    for (int q = 0; q < SB::kN; ++q) {
      if constexpr (KB) {
        R.b[q] = piece_of<E, ANY>(bp[q] + static_cast<size_t>(st) * 128, g.K - k0 - bpiece * I::kPiece);
      } else if constexpr (PAIR) {
        const int k = k0 + brow + SB::kStep * q, kk = k < g.b.half ? k : k - g.b.half;
        const uint8_t* base = static_cast<const uint8_t*>(k < g.b.half ? g.b.p : g.b.q);
        const bool ok = k < g.K && kk < g.b.live;
        R.b[q] = piece_of<E, ANY>(base + (static_cast<size_t>(kk) * g.b.ld + n0) * I::kSize + 16 * bpiece, ok ? bleft : 0);
      } else {
        const bool ok = k0 + brow + SB::kStep * q < g.K;
        R.b[q] = piece_of<E, ANY>(bp[q] + static_cast<size_t>(k0) * g.b.ld * I::kSize, ok ? bleft : 0);
      }
    }
  };
  const uint32_t alds = arow * SA::kRow + (KA ? ((apiece ^ ((arow >> 1) & 7)) * 16) : 16 * apiece);
  const uint32_t blds = SA::kBytes + brow * SB::kRow + (KB ? ((bpiece ^ ((brow >> 1) & 7)) * 16) : 16 * bpiece);
  auto store = [&](const Regs& R, int buf) __attribute__((always_inline)) {
    uint8_t* d = smem + buf * kStageBytes;
#pragma unroll
    for (int q = 0; q < SA::kN; ++q) *reinterpret_cast<uint4*>(d + alds + q * SA::kStep * SA::kRow) = R.a[q];
#pragma unroll
    for (int q = 0; q < SB::kN; ++q) *reinterpret_cast<uint4*>(d + blds + q * SB::kStep * SB::kRow) = R.b[q];
  };
  Acc<E> acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  // Fragment kk of the 32 rows from row on: 16 bytes of contraction of the lane's row, the
  // same elements of either operand for a lane half.
  const uint32_t swz = static_cast<uint32_t>(hi ^ ((r32 >> 1) & 7));
  auto frag = [&](auto side, const uint8_t* base, int row, int kk, bool kc) __attribute__((always_inline)) {
    using S = decltype(side);
    if (kc) return *reinterpret_cast<const uint4*>(base + (row + r32) * 128 + ((2 * kk) ^ swz) * 16);
    if constexpr (E == El::BF16) {
      const uint8_t* t = base + (16 * kk + 8 * hi + ((lane & 15) >> 2)) * S::kRow + (row + (r32 & 16) + 4 * (lane & 3)) * 2;
      const uint2 lo = lds_turned(t), up = lds_turned(t + 4 * S::kRow);
      return uint4{lo.x, lo.y, up.x, up.y};
    } else {
      const uint8_t* t = base + (8 * kk + 4 * hi) * S::kRow + (row + r32) * 4;
      return uint4{*reinterpret_cast<const uint32_t*>(t), *reinterpret_cast<const uint32_t*>(t + S::kRow),
                   *reinterpret_cast<const uint32_t*>(t + 2 * S::kRow), *reinterpret_cast<const uint32_t*>(t + 3 * S::kRow)};
    }
  };
  auto compute = [&](int buf) __attribute__((always_inline)) {
    const uint8_t* As = smem + buf * kStageBytes;
    const uint8_t* Bs = As + SA::kBytes;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint4 af[NI], bf[NJ];
#pragma unroll
      for (int i = 0; i < NI; ++i) af[i] = frag(SA{}, As, wm * (BM / 2) + 32 * i, kk, KA);
#pragma unroll
      for (int j = 0; j < NJ; ++j) bf[j] = frag(SB{}, Bs, wn * (BN / 2) + 32 * j, kk, KB);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma32<E>(af[i], bf[j], acc[i][j]);
    }
  };

  // This part's full stages: the f'th is lo + f, or, from n0f on, lo2 + f - n0f.
  const int lo = min(s0, full), n_lo = max(min(s1, full) - lo, 0), lo2 = max(s0, up), n_up = max(min(s1, up + full) - lo2, 0);
  const int n_full = n_lo + n_up;
  auto full_at = [&](int f) { const int t = min(f, n_full - 1); return t < n_lo ? lo + t : lo2 + t - n_lo; };
  // Iteration f: barrier; write full stage f + 1 from registers, start loading f + 1 + kDepth
  // into them (past the end the last one again), multiply f.  Small tiles, which are few
  // when the product is, have more stages on their way.
  constexpr int kDepth = BM * BN > 64 * 64 ? 2 : 4;
  if (n_full > 0) {
    Regs R[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load_full(R[d], full_at(d));
    store(R[0], 0);
    load_full(R[0], full_at(kDepth));
    for (int f = 0; f < n_full; f += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (f + d >= n_full) break;
        __syncthreads();
        store(R[(d + 1) % kDepth], (d + 1) & 1);
        load_full(R[(d + 1) % kDepth], full_at(f + d + 1 + kDepth));
        compute(d & 1);
      }
    }
  }
  // The others, one at most but for a pair, for which there are at most two of either half.
  for (int st = s0; st < s1; ++st) {
    if (st < full || (st >= up && st < up + full)) {
      st = (st < full ? full : up + full) - 1;
      continue;
    }
    Regs R;
    load_part(R, st);
    __syncthreads();
    store(R, 0);
    __syncthreads();
    compute(0);
  }

  // Out through LDS, NI rounds of 32 rows of each wave row, rows padded by 8 floats.
  // Lane l, element v: row 8 (v / 4) + 4 (l / 32) + v % 4, column l % 32 of a block.
  float* stg = reinterpret_cast<float*>(smem);
  const int n = n0 + 4 * (tid % (kCols / 4));
  const auto row_of = [&](int R) { return m0 + (R >> 5 & 1) * (BM / 2) + 32 * (R >> 6) + (R & 31); };
  typename Epi::Cols cols;
  constexpr int kRows = kCols / 16 < 4 ? kCols / 16 : 4;         // of a batch
  Batch<Epi, kRows> ahead;
  if (parts == 1 && n < g.N) {
    cols = epi.cols(n);
    ahead.load(epi, g.M, n, tid / (kCols / 4), 256 / (kCols / 4), row_of);
  }
  // A part: M rows of the first product's columns, then M of the second's.
  const size_t np = part_stride(g.N), second = static_cast<size_t>(g.M) * np;
  const auto part_of = [&](int R) {
    const int m = row_of(R);
    return m < g.M ? part + (static_cast<size_t>(p) * g.M * (kPair ? 2 : 1) + m) * np + n : nullptr;
  };
  __syncthreads();                   // every wave is done reading the stage buffers
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        stg[(wm * 32 + 8 * (v >> 2) + 4 * hi + (v & 3)) * kStride + wn * (BN / 2) + 32 * j + r32] = as_float(acc[i][j][v]);
    __syncthreads();
    results_out<E, kPair, kTurn, BN, 64, 256, kRows>(g, epi, cols, ahead, stg, kStride, n, tid, 64 * i, i + 1 < NI, row_of, parts > 1, part_of, second);
    __syncthreads();
  }
}

// ---------------------------------------------------------------- at most 16 rows
//
// The weights go from memory straight into the registers of the MFMAs (skinny.h): eight
// waves compute 8 SETS operand columns over one part of the contraction, an eighth for
// each.  Of a pair the two sets are eight columns of either product.
//
// Bound by memory: one row against the two bf16 matrices of 17408 x 5120 takes 64 us
// (5.5 TB/s), against the third 39 (4.5 TB/s; 640 workgroups only); 17408 x 5120 int8 21 to
// 22 us (4.1 TB/s).  With 16 rows the rows' own reading, by every workgroup, shows: the three
// matrices take 163 us instead of 103.
constexpr int kSkinnyEight = 8;

template <El E>
using Acc16 = std::conditional_t<E == El::I8, i32x4v, f32x4>;
template <El E>
__device__ __forceinline__ Acc16<E> mfma16(const uint4& a, const uint4& b, Acc16<E> c) {
  if constexpr (E == El::F32) {
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  } else if constexpr (E == El::BF16) {
    return mfma_bf16_16x16x32(a, b, c);
  } else {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4v, a), __builtin_bit_cast(i32x4v, b), c, 0, 0, 0);
  }
}

// Where the rows of x come from: as they lie, as operands; at most eight, with what their
// rounding left eight rows further on, which takes the place of the tile's idle rows; or a
// single row that a functor puts into LDS once the first weights are on their way; it also
// gives what the epilogue reads of that row.
struct AsTheyLie {
  static constexpr bool kStaged = false, kRests = false;
};
struct WithRests {
  static constexpr bool kStaged = false, kRests = true;
};
constexpr int kRestRows = 8;

template <El E, bool PAIR, bool ANY, int SETS, class Rows, class Epi>
__global__ void __launch_bounds__(kSkinnyEight * kWave, SETS == 1 ? 6 : 4) product_skinny_kernel(Product g, Rows rows, Epi epi, int parts, float* part) {
  using I = ElInfo<E>;
  static_assert(!PAIR || SETS == 2, "a set for either product");
  constexpr int kCols = PAIR ? 8 : 8 * SETS, D = SETS == 1 ? 4 : 5;
  __shared__ f32x4 red[kSkinnyEight][kWave];
  __shared__ __attribute__((aligned(16))) float out[16][20];      // read by fours
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * kCols, p = blockIdx.y;
  const int nb = static_cast<int>(ceil_div(g.K, I::kStage));
  const int b0 = static_cast<int>(static_cast<int64_t>(p) * nb / parts), b1 = static_cast<int>(static_cast<int64_t>(p + 1) * nb / parts);
  const int lo = b0 + wave * (b1 - b0) / kSkinnyEight, hi = b0 + (wave + 1) * (b1 - b0) / kSkinnyEight;
  const uint8_t* wbase[SETS];
  uint32_t woff[SETS];
#pragma unroll
  for (int h = 0; h < SETS; ++h) {
    wbase[h] = static_cast<const uint8_t*>(PAIR && h ? g.b.q : g.b.p) + static_cast<size_t>(n0) * g.b.ld * I::kSize;
    woff[h] = static_cast<uint32_t>(min((PAIR ? 0 : 8 * h) + (lane & 7), g.N - 1 - n0)) * static_cast<uint32_t>(g.b.ld) * I::kSize + 16 * lane_piece(lane);
  }
  const uint8_t* xbase = static_cast<const uint8_t*>(g.a.p);
  const bool live = (Rows::kRests ? r & 7 : r) < g.M;
  const uint32_t xoff = static_cast<uint32_t>(live ? r : 0) * static_cast<uint32_t>(g.a.ld) * I::kSize + 16 * q;
  const bool tail = g.K % I::kStage != 0;
  extern __shared__ __attribute__((aligned(16))) uint8_t staged[];

  struct Blk {
    uint4 w[SETS], x[Rows::kStaged ? 1 : 2];
  };
  Acc16<E> acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  int at = lo, use = lo;
  batches<D, Blk>(
      hi - lo,
      [&](Blk& k) __attribute__((always_inline)) {
        const size_t o = static_cast<size_t>(at) * 128;
        const int left = g.K - at * I::kStage;     // elements from this block on; only the last can be cut
        if constexpr (!Rows::kStaged) k.x[0] = k.x[1] = uint4{0, 0, 0, 0};
        if (!ANY && !tail) {
#pragma unroll
          for (int h = 0; h < SETS; ++h) k.w[h] = ld16_stream(wbase[h] + o + woff[h]);
          if constexpr (!Rows::kStaged) {
            if (live) {
              k.x[0] = ld16(xbase + o + xoff);
              k.x[1] = ld16(xbase + o + xoff + 64);
            }
          }
        } else {
#pragma unroll
          for (int h = 0; h < SETS; ++h) k.w[h] = piece_of<E, ANY>(wbase[h] + o + woff[h], left - I::kPiece * lane_piece(lane));
          if constexpr (!Rows::kStaged) {
            if (live) {
              k.x[0] = piece_of<E, ANY>(xbase + o + xoff, left - I::kPiece * q);
              k.x[1] = piece_of<E, ANY>(xbase + o + xoff + 64, left - I::kPiece * (q + 4));
            }
          }
        }
        ++at;
      },
      [&](Blk& k) __attribute__((always_inline)) {
        uint4 x[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        if constexpr (Rows::kStaged) {
          if (live) {
            const uint8_t* b = staged + use * 128 + 16 * q;
            x[0] = *reinterpret_cast<const uint4*>(b);
            x[1] = *reinterpret_cast<const uint4*>(b + 64);
          }
          ++use;
        } else {
          x[0] = k.x[0];
          x[1] = k.x[1];
        }
        if constexpr (SETS == 2) {
          const bool upper = lane & 8;
          trade(k.w[0].x, k.w[1].x, upper);
          trade(k.w[0].y, k.w[1].y, upper);
          trade(k.w[0].z, k.w[1].z, upper);
          trade(k.w[0].w, k.w[1].w, upper);
          acc[0] = mfma16<E>(x[0], k.w[0], acc[0]);
          acc[0] = mfma16<E>(x[1], k.w[1], acc[0]);
        } else {
          acc[0] = mfma16<E>(x[0], k.w[0], acc[0]);
          acc[1] = mfma16<E>(x[1], k.w[0], acc[1]);
        }
      },
      [&] {
        if constexpr (Rows::kStaged) rows.put(staged, g.K, blockIdx.x == 0 && p == 0);
      });
  f32x4 s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (SETS == 2) {
      s[i] = as_float(acc[0][i]);
    } else {
      // Eight columns: the halves of a block were multiplied over all sixteen, of which the
      // lower eight are the first half's and the upper eight the second's.
      const auto v = (lane & 8) ? acc[1][i] : acc[0][i];
      s[i] = as_float(v + __shfl_xor(v, 8, kWave));
    }
  }
  red[wave][lane] = s;
  __syncthreads();
  // Wave w < 4 adds elements i = w: rows 4 q + w.
  if (wave < 4) {
    float v = red[0][lane][wave];
#pragma unroll
    for (int o = 1; o < kSkinnyEight; ++o) v = add_sums<E>(v, red[o][lane][wave]);
    out[4 * q + wave][r] = v;
  }
  __syncthreads();
  constexpr int kQuads = kCols / 4;
  const int m = tid / kQuads, c = 4 * (tid % kQuads), n = n0 + c;
  if (m >= g.M || n >= g.N) return;
  f32x4 a = *reinterpret_cast<const f32x4*>(&out[m][c]);
  if constexpr (Rows::kRests) {
    // Beside an infinity a rest says nothing: a rest of 0 or of the other sign meets an infinite
    // weight as NaN or as the other infinity.
    const f32x4 b = *reinterpret_cast<const f32x4*>(&out[m + kRestRows][c]);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = isfinite(a[e]) ? a[e] + b[e] : a[e];
  }
  f32x4 u = {0.f, 0.f, 0.f, 0.f};
  if constexpr (PAIR) u = *reinterpret_cast<const f32x4*>(&out[m][c + 8]);
  if (parts > 1) {
    const size_t np = part_stride(g.N), o = (static_cast<size_t>(p) * g.M * (PAIR ? 2 : 1) + m) * np + n;
    *reinterpret_cast<f32x4*>(part + o) = a;
    if constexpr (PAIR) *reinterpret_cast<f32x4*>(part + o + g.M * np) = u;
  } else {
    if constexpr (Rows::kStaged) epi.put(m, n, whole_sums<E>(a), u, epi.cols(n), rows.ahead(staged, epi, n));
    else epi.put(m, n, whole_sums<E>(a), u, epi.cols(n), epi.ahead(m, n));
  }
}

// ---------------------------------------------------------------- aligned tiles
//
// BM x BN sums per workgroup of 2 x 2 waves, for operands in whole 16-byte pieces (bf16 and
// 8-bit).  In 256 x 256 tiles a wave computes 128 x 128, alone on its SIMD: a stage's
// fragments leave LDS twice, not three times as with eight waves of 128 x 64.  A stage is
// 64 bf16 (128 int8) of contraction and goes to one of BUFS buffers in LDS by DMA.  Nothing
// but a wave's own instructions hides its latencies: the fragments of a quarter stage are
// read while the quarter before is multiplied, across the stages' border too; the DMA of A
// of stage s + BUFS is issued in the last quarter of s and that of B in the first of s + 1
// (both in one quarter fill the queue and hold up the MFMAs: 8 % slower).  One barrier a
// stage, in front of the last quarter: by then every wave has the stage's last fragments in
// registers and stage s + 1 is in LDS.
//
// Bound by the matrix cores, whose clock falls under full load: they are busy 78 % of the
// 256 x 256 kernel's time, at 1.8 GHz.  8192 x 17408 x 5120 bf16 with a pair takes 2.36 to 2.48 ms
// (1.18 to 1.24 PFLOP/s, its results included), one product of these sizes 1.11 to 1.14
// (1.28 to 1.32; a library product without an epilogue 1.20, or 1.39 with a k-strided side);
// 8192 x 4096 x 7168 int8 221 to 255 us (1.9 to 2.2 POP/s; a library product 204).
//
// k-contiguous operands: rows of 128 bytes, 16-byte pieces permuted by (row / 2) mod 8.
// k-strided: a row for each k, 64-byte pieces permuted by k mod 4, so that the four k of a
// turning read lie in different quarters of the banks.  What lies behind the end of the
// contraction is out of the resource's range, and such loads bring zeros.
//
// Results leave through LDS too, 32 rows of a wave at a time, in a buffer that the last
// stage is not in, the first or the last; rows padded by 4 floats, for which there is room
// on its other side.
template <El E, bool KA, bool KB, bool PAIR, int BM, int BN, int BUFS>
struct Aligned {
  static constexpr bool kPair = PAIR && KB;
  static constexpr int kCols = kPair ? BN / 2 : BN;
  static constexpr int kSideA = BM * 128, kStage = (BM + BN) * 128;
  static constexpr int kOut = BN / 2 + 4, kStaged = 4 * 32 * kOut * 4;
  static constexpr int kPad = kStaged > kStage ? (kStaged - kStage + 1023) / 1024 * 1024 : 0, kLds = BUFS * kStage + 2 * kPad;
  // Tiles that run on a CU at a time, by the LDS.
  static constexpr int kOnCu = 2 * kLds <= (160 << 10) ? 2 : 1;
  static_assert(BM > 64 || KA, "the banks of a k-strided side need 128 columns");
  static constexpr int kBand = 2048 / BM;        // row blocks of a band of tiles
};

// One instruction: lane l loads 16 bytes at voff to LDS at lds + 16 l, zeros out of range.
// (No scalar offset: the range check takes it off the range.)
__device__ __forceinline__ void dma_line(i32x4_t rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %[lds]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v], %[rs], 0 offen lds"
               :
               : [v] "v"(voff), [rs] "s"(rsrc), [lds] "s"(lds)
               : "memory");
}

// What a wave loads of one operand: kN instructions a stage.
template <El E, bool KC, bool PAIR, int R>
struct AlignedSide {
  using I = ElInfo<E>;
  static constexpr int kN = R / 32;
  static constexpr int kLanes = R * I::kSize / 16, kStep = 64 / kLanes;   // k-strided: lanes of a k, k of an instruction
  static constexpr uint32_t kNowhere = 0x80000000u;                       // out of any range
  const uint8_t *p, *q;          // the tile's first row (k-contiguous) or column (k-strided), k = 0
  uint32_t ld, bytes;            // of a row or k; k-contiguous: of the tile's part of a stage
  uint32_t voff[kN];
  int last;                      // k-strided: the last 16-byte piece of the tile's columns
  int piece;                     // k-contiguous: the lane's piece of rows of even instructions; odd ones ^ 4
  int K, half, live;
  __device__ __forceinline__ AlignedSide(const Operand& o, int r0, int rows, int k, int wave, int lane) {
    ld = static_cast<uint32_t>(o.ld) * I::kSize;
    K = k;
    half = o.half;
    live = o.live;
    if constexpr (KC) {
      last = min(PAIR ? R / 2 : R, rows - r0) - 1;
      p = static_cast<const uint8_t*>(o.p) + static_cast<size_t>(r0) * ld;
      q = PAIR ? static_cast<const uint8_t*>(o.q) + static_cast<size_t>(r0) * ld : nullptr;
      bytes = static_cast<uint32_t>(last) * ld + 128;
      piece = (lane & 7) ^ (lane >> 4);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int r = R / 4 * wave + 8 * i + (lane >> 3), row = PAIR ? (r >> 6) * 32 + (r & 31) : r;
        voff[i] = static_cast<uint32_t>(min(row, last)) * ld + (piece ^ (i & 1) * 4) * 16;
      }
    } else {
      p = static_cast<const uint8_t*>(o.p) + static_cast<size_t>(r0) * I::kSize;
      q = PAIR ? static_cast<const uint8_t*>(o.q) + static_cast<size_t>(r0) * I::kSize : nullptr;
      last = min(R, rows - r0) / I::kPiece - 1;
      // Instructions of a stage repeat after two (two k each) or one (four k).
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k0 = lane / kLanes, s = (kStep * i + k0) & 3;
        voff[i] = static_cast<uint32_t>(I::kStage / 4 * wave + k0) * ld + min((lane % kLanes) ^ (s << 2), last) * 16;
      }
    }
  }
  // The resource of stage ks, and of the pair's second matrix.
  __device__ __forceinline__ i32x4_t rsrc(int ks, bool second = false) const {
    if constexpr (KC) {
      return dma_rsrc((PAIR && second ? q : p) + static_cast<size_t>(ks) * 128, bytes);
    } else {
      const bool up = PAIR && ks * I::kStage >= half;
      const int k = ks * I::kStage - (up ? half : 0), left = min((PAIR ? live : K) - k, I::kStage);
      return dma_rsrc((up ? q : p) + static_cast<size_t>(max(min(k, (PAIR ? live : K) - 1), 0)) * ld,
                      left > 0 ? static_cast<uint32_t>(left - 1) * ld + static_cast<uint32_t>(last + 1) * 16 : 0u);
    }
  }
  // k-contiguous: before the last stage, if it is cut, its pieces past the end go nowhere.
  __device__ __forceinline__ void cut(int ks) {
    if constexpr (KC) {
      const int left = (K - ks * I::kStage) / I::kPiece;
      if (left >= 8) return;
#pragma unroll
      for (int i = 0; i < kN; ++i) voff[i] += (piece ^ (i & 1) * 4) < left ? 0u : kNowhere;
    }
  }
  __device__ __forceinline__ void issue(const i32x4_t& r, int i, uint32_t lds) const {
    if constexpr (KC) dma_line(r, voff[i], lds + 1024 * i);
    else dma_line(r, voff[kStep == 2 ? i & 1 : 0] + ld * (kStep * i), lds + 1024 * i);
  }
  // Whether instruction i of the wave loads rows of the pair's second matrix.
  static __device__ __forceinline__ bool second(int wave, int i) { return (R / 4 * wave + 8 * i) >> 5 & 1; }
};

// Tiles are walked in bands of 2048 rows, so that the tiles that run on an XCD at a time
// share few row and column blocks in its L2.
template <int BM, int BAND, int COLS>
__device__ __forceinline__ void tile_place(int tile, int mt, int nt, int& m0, int& n0) {
  const int band = tile / (BAND * nt), in_band = tile - band * BAND * nt;
  const int bm = min(BAND, mt - band * BAND);
  m0 = (band * BAND + in_band % bm) * BM;
  n0 = in_band / bm * COLS;
}

template <El E, bool KA, bool KB, bool PAIR, int BM, int BN, int BUFS, class Epi>
__global__ void __launch_bounds__(256, (Aligned<E, KA, KB, PAIR, BM, BN, BUFS>::kOnCu)) product_aligned_kernel(Product g, Epi epi, int whole, int parts, float* part) {
  using L = Aligned<E, KA, KB, PAIR, BM, BN, BUFS>;
  constexpr bool kPair = L::kPair;
  constexpr int kCols = L::kCols, NI = BM / 64, NJ = BN / 64;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[L::kLds];
  uint8_t* smem = lds + L::kPad;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hi = lane >> 5;
  const int mt = static_cast<int>(ceil_div(g.M, BM)), nt = static_cast<int>(ceil_div(g.N, kCols));
  const int stages = static_cast<int>(ceil_div(g.K, ElInfo<E>::kStage));
  using SideA = AlignedSide<E, KA, false, BM>;
  using SideB = AlignedSide<E, KB, PAIR, BN>;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(smem));
  const uint32_t lds_a = lds0 + SideA::kN * 1024 * wave, lds_b = lds0 + L::kSideA + SideB::kN * 1024 * wave;

  // Offsets of the wave's fragments in a side: k-contiguous by quarter (block x is 4 KiB
  // on), k-strided by block (quarter kk is 16 rows on).
  constexpr int kRowA = BM * ElInfo<E>::kSize, kRowB = BN * ElInfo<E>::kSize;
  uint32_t fa[4], fb[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t kc = static_cast<uint32_t>(r32 * 128 + (((2 * x) ^ hi ^ ((r32 >> 1) & 7)) * 16));
    const uint32_t s = (lane & 15) >> 2, in = (r32 & 16) * 2 + 8 * (lane & 3);
    fa[x] = KA ? kc + wm * BM / 2 * 128 : (8 * hi + s) * kRowA + ((wm * NI + x) ^ s) * 64 + in;
    fb[x] = L::kSideA + (KB ? kc + wn * BN / 2 * 128 : (8 * hi + s) * kRowB + ((wn * NJ + x) ^ s) * 64 + in);
  }
  auto frag = [&](const uint8_t* base, const uint32_t (&f)[4], int blk, int kk, auto kc, auto row) __attribute__((always_inline)) {
    if constexpr (decltype(kc)::value) {
      return *reinterpret_cast<const uint4*>(base + f[kk] + blk * 4096);
    } else {
      const uint8_t* t = base + f[blk] + kk * 16 * decltype(row)::value;
      const uint2 lo = lds_turned(t), up = lds_turned(t + 4 * decltype(row)::value);
      return uint4{lo.x, lo.y, up.x, up.y};
    }
  };
  auto frag_a = [&](const uint8_t* base, int i, int kk) __attribute__((always_inline)) {
    return frag(base, fa, i, kk, std::bool_constant<KA>{}, std::integral_constant<int, kRowA>{});
  };
  auto frag_b = [&](const uint8_t* base, int j, int kk) __attribute__((always_inline)) {
    return frag(base, fb, j, kk, std::bool_constant<KB>{}, std::integral_constant<int, kRowB>{});
  };
  using Yes = std::true_type;
  using No = std::false_type;

  // Workgroup b runs on XCD b % 8 and takes every step'th of that XCD's share of the whole
  // tiles, which come in full rounds; then one of its share of the rest, in parts.
  const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3, step = gridDim.x >> 3;
  const int rest = (mt * nt - whole) * parts, share = whole / 8, rest_share = (rest + 7) / 8;
  for (int turn = at; turn < share + step; turn += step) {
    int tile, p = 0, cut = 1;
    if (turn < share) {
      tile = xcd * share + turn;
    } else {
      const int item = xcd * rest_share + at;
      if (at >= rest_share || item >= rest) break;
      tile = whole + item / parts;
      p = item % parts;
      cut = parts;
    }
    const int k0 = static_cast<int>(static_cast<int64_t>(p) * stages / cut), nk = static_cast<int>(static_cast<int64_t>(p + 1) * stages / cut);
    int m0, n0;
    tile_place<BM, L::kBand, kCols>(tile, mt, nt, m0, n0);
    SideA A(g.a, m0, g.M, g.K, wave, lane);
    SideB B(g.b, n0, g.N, g.K, wave, lane);
    auto dma_a = [&](int ks, uint32_t buf) __attribute__((always_inline)) {
      const i32x4_t r = A.rsrc(ks);
      A.cut(ks);
#pragma unroll
      for (int i = 0; i < SideA::kN; ++i) A.issue(r, i, lds_a + buf);
    };
    auto dma_b = [&](int ks, uint32_t buf) __attribute__((always_inline)) {
      const i32x4_t r = B.rsrc(ks), r2 = kPair ? B.rsrc(ks, true) : r;
      B.cut(ks);
#pragma unroll
      for (int i = 0; i < SideB::kN; ++i) B.issue(kPair && SideB::second(wave, i) ? r2 : r, i, lds_b + buf);
    };
    constexpr int kLoads = SideA::kN + SideB::kN;     // of a stage
    __syncthreads();                 // the tile before is done with LDS
    // BUFS - 1 stages and A of the next, as far as there are any.
#pragma unroll
    for (int d = 0; d < BUFS; ++d)
      if (k0 + d < nk) {
        dma_a(k0 + d, d * L::kStage);
        if (d < BUFS - 1) dma_b(k0 + d, d * L::kStage);
      }
    if (k0 + BUFS <= nk) wait_vm<(BUFS - 2) * kLoads + SideA::kN>();
    else wait_vm<0>();
    __syncthreads();
    Acc<E> acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    uint4 af[2][NI], bf[2][NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) bf[0][j] = frag_b(smem, j, 0);
#pragma unroll
    for (int i = 0; i < NI; ++i) af[0][i] = frag_a(smem, i, 0);
    // The MFMAs of quarter kk, by twos; between them the fragments of the quarter after it
    // (`read`) and `n` instructions of a stage's DMA.
    constexpr int kPairs = NI * NJ / 2;
    auto quarter = [&](int kk, const uint8_t* next, int nkk, auto read, auto n, auto dma) __attribute__((always_inline)) {
      const int c = kk & 1, d = c ^ 1;
#pragma unroll
      for (int x = 0; x < kPairs; ++x) {
        if constexpr (decltype(read)::value) {
#pragma unroll
          for (int y = x * (NI + NJ) / kPairs; y < (x + 1) * (NI + NJ) / kPairs; ++y) {
            if (y < NJ) bf[d][y] = frag_b(next, y, nkk);
            else af[d][y - NJ] = frag_a(next, y - NJ, nkk);
          }
        }
#pragma unroll
        for (int y = x * decltype(n)::value / kPairs; y < (x + 1) * decltype(n)::value / kPairs; ++y) dma(y);
        const int i = 2 * x / NJ, j = 2 * x % NJ;
        acc[i][j] = mfma32<E>(bf[c][j], af[c][i], acc[i][j]);
        acc[i][j + 1] = mfma32<E>(bf[c][j + 1], af[c][i], acc[i][j + 1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    const auto nothing = [](int) __attribute__((always_inline)) {};
    using Zero = std::integral_constant<int, 0>;
    // Stage ks in the buffer at `buf`; B of stage ks + BUFS - 1 and A of stage ks + BUFS are
    // loaded meanwhile, where they are (`last`: there is no stage ks + 1 either).
    uint32_t buf = 0;
    auto stage = [&](int ks, auto load_b, auto load_a, auto last) __attribute__((always_inline)) {
      const uint32_t next = buf + L::kStage == BUFS * L::kStage ? 0 : buf + L::kStage;
      const uint32_t before = buf == 0 ? (BUFS - 1) * L::kStage : buf - L::kStage;
      const uint8_t* here = smem + buf;
      if constexpr (decltype(load_b)::value) {
        const i32x4_t r = B.rsrc(ks + BUFS - 1), r2 = kPair ? B.rsrc(ks + BUFS - 1, true) : r;
        B.cut(ks + BUFS - 1);
        quarter(0, here, 1, Yes{}, std::integral_constant<int, SideB::kN>{}, [&](int i) __attribute__((always_inline)) {
          B.issue(kPair && SideB::second(wave, i) ? r2 : r, i, lds_b + before);
        });
      } else {
        quarter(0, here, 1, Yes{}, Zero{}, nothing);
      }
      quarter(1, here, 2, Yes{}, Zero{}, nothing);
      quarter(2, here, 3, Yes{}, Zero{}, nothing);
      if constexpr (!decltype(last)::value) {
        // The stage's last fragments are in registers, the next stage is in LDS; the stages
        // behind it may still be on their way.
        if constexpr (decltype(load_b)::value) wait_vm<(BUFS - 2) * kLoads>();
        else wait_vm<0>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const uint8_t* there = smem + next;
        if constexpr (decltype(load_a)::value) {
          const i32x4_t r = A.rsrc(ks + BUFS);
          A.cut(ks + BUFS);
          quarter(3, there, 0, Yes{}, std::integral_constant<int, SideA::kN>{}, [&](int i) __attribute__((always_inline)) {
            A.issue(r, i, lds_a + buf);
          });
        } else {
          quarter(3, there, 0, Yes{}, Zero{}, nothing);
        }
        buf = next;
      } else {
        quarter(3, here, 0, No{}, Zero{}, nothing);
      }
    };
    int ks = k0;
    for (; ks + BUFS < nk; ++ks) stage(ks, Yes{}, Yes{}, No{});
    if (ks + BUFS == nk) stage(ks++, Yes{}, No{}, No{});
    for (; ks + 1 < nk; ++ks) stage(ks, No{}, No{}, No{});
    stage(ks, No{}, No{}, Yes{});

    // Lane l, element v of a block (the operands' roles are exchanged): row l % 32, column
    // 8 (v / 4) + 4 (l / 32) + v % 4.  A wave's staged rows are its own.
    constexpr int kWaveCols = kCols / 2, kLanes = kWaveCols / 4;
    constexpr int kAhead = Epi::kAhead < 32 / (64 / kLanes) ? Epi::kAhead : 32 / (64 / kLanes);
    const uint32_t free_buf = buf ? 0 : L::kPad + (BUFS - 1) * L::kStage;     // the first or the last
    float* stg = reinterpret_cast<float*>(lds + free_buf) + wave * 32 * L::kOut;
    const int c = 4 * (lane % kLanes), n = n0 + wn * kWaveCols + c;
    const int staged = kPair ? (c >> 5) * 64 + (c & 31) : c;
    const auto row_of = [&](int R) { return m0 + wm * (BM / 2) + R; };
    float* mine = part + ((static_cast<size_t>(tile - whole) * parts + p) * BM + wm * (BM / 2)) * BN + wn * (BN / 2) + staged;
    typename Epi::Cols cols;
    Batch<Epi, kAhead> ahead;
    if (cut == 1 && n < g.N) {
      cols = epi.cols(n);
      ahead.load(epi, g.M, n, lane / kLanes, 64 / kLanes, row_of);
    }
    auto stage_rows = [&](const Acc<E> (&r)[NJ]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = as_float(r[j][4 * q + e]);
          *reinterpret_cast<f32x4*>(stg + r32 * L::kOut + 32 * j + 8 * q + 4 * hi) = v;
        }
    };
    // One copy of the epilogue for all blocks of rows: unrolled, its activations do not fit
    // the instruction cache.
#pragma unroll 1
    for (int i = 0; i < NI; ++i) {
      if (i == 0) stage_rows(acc[0]);
      if constexpr (NI > 1)
        if (i == 1) stage_rows(acc[1]);
      if constexpr (NI > 2) {
        if (i == 2) stage_rows(acc[2]);
        if (i == 3) stage_rows(acc[3]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      results_out<E, kPair, 32, BN / 2, 32, 64, kAhead>(g, epi, cols, ahead, stg, L::kOut, n, lane, 32 * i, i + 1 < NI, row_of,
                                                    cut > 1, [&](int R) { return mine + R * BN; }, 32);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// The rest's parts added in order: 1024 sums (of a pair: 512 of either) to a workgroup.
template <El E, bool PAIR, int BM, int BN, class Epi>
__global__ void __launch_bounds__(256) product_rest_kernel(Product g, Epi epi, int whole, int parts, const float* part) {
  constexpr int kCols = PAIR ? BN / 2 : BN, kQuads = kCols / 4, kGroups = BM * kQuads / 256, kBand = 2048 / BM;
  const int mt = static_cast<int>(ceil_div(g.M, BM)), nt = static_cast<int>(ceil_div(g.N, kCols));
  const int tile = blockIdx.x / kGroups, i = (blockIdx.x % kGroups) * 256 + threadIdx.x;
  int m0, n0;
  tile_place<BM, kBand, kCols>(whole + tile, mt, nt, m0, n0);
  const int R = i / kQuads, c = 4 * (i % kQuads), m = m0 + R, n = n0 + c;
  if (m >= g.M || n >= g.N) return;
  const typename Epi::Cols cols = epi.cols(n);
  const typename Epi::Ahead ahead = epi.ahead(m, n);
  const float* q = part + (static_cast<size_t>(tile) * parts * BM + R) * BN + (PAIR ? (c >> 5) * 64 + (c & 31) : c);
  f32x4 s = {0.f, 0.f, 0.f, 0.f}, u = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; p += kSumAhead) {
    f32x4 b[kSumAhead], d[kSumAhead];
#pragma unroll
    for (int k = 0; k < kSumAhead; ++k)
      if (p + k < parts) {
        b[k] = *reinterpret_cast<const f32x4*>(q + static_cast<size_t>(p + k) * BM * BN);
        if constexpr (PAIR) d[k] = *reinterpret_cast<const f32x4*>(q + static_cast<size_t>(p + k) * BM * BN + 32);
      }
#pragma unroll
    for (int k = 0; k < kSumAhead; ++k)
      if (p + k < parts)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[e] = add_sums<E>(s[e], b[k][e]);
          if constexpr (PAIR) u[e] += d[k][e];
        }
  }
  epi.put(m, n, whole_sums<E>(s), u, cols, ahead);
}

// ---------------------------------------------------------------- host

constexpr int kCus = 256;
constexpr int kMaxParts = 16;
// Most bytes of partial sums: those of a 256 x 256 tile on each CU.
constexpr size_t kMaxPartBytes = size_t{kCus} * 256 * 256 * sizeof(float);
// Bytes of partial sums of any product of at most M rows.
inline size_t part_bytes(bool pair, int64_t M, int64_t N) {
  const double want = static_cast<double>(kMaxParts) * M * (pair ? 2 : 1) * part_stride(N) * sizeof(float);
  return want < static_cast<double>(kMaxPartBytes) ? std::max<size_t>(align_up(static_cast<size_t>(want), 256), 256) : kMaxPartBytes;
}

struct TilePlan {
  int rows, cols;       // of a tile, in operand rows
  int bufs;             // of the DMA kernel, 0: any alignment
  int64_t tiles;
  int64_t whole;        // aligned: tiles that are not cut
  int parts;            // of the others
};

// The cheapest tile and split by an estimate in microseconds: what a CU takes in (28 KB a
// microsecond with two tiles on it, 20 with one), the f32 matrix rate, and the partial sums'
// way out and back.
inline TilePlan plan_tiles(El e, bool pair, int out_bytes, bool by_dma, bool strided, int64_t M, int64_t N, int64_t K) {
  const int size = e == El::F32 ? 4 : e == El::BF16 ? 2 : 1;
  const int64_t width = pair ? 2 * N : N, stages = ceil_div(K * size, 128);
  const double room = static_cast<double>(part_bytes(pair, M, N));
  TilePlan best{};
  double least = 0;
  const auto offer = [&](double us, const TilePlan& t) {
    if (best.tiles && us >= least) return;
    least = us;
    best = t;
  };
  static const struct { int rows, cols; } kTiles[] = {{64, 64}, {64, 128}, {128, 128}};
  for (const auto& t : kTiles) {
    if (t.cols == 64 && e != El::F32) continue;
    const int64_t tiles = ceil_div(M, t.rows) * ceil_div(width, t.cols), slots = int64_t{2} * kCus;
    for (int parts = 1; parts <= kMaxParts; ++parts) {
      const double planes = static_cast<double>(parts) * M * (pair ? 2 : 1) * part_stride(N) * 4;
      if (parts > 1 && (tiles * parts > (e == El::F32 ? 2 * slots : slots) || planes > room || stages / parts < 4)) break;
      const int64_t items = tiles * parts, rounds = ceil_div(items, slots);
      const double shared = items > kCus ? 2 : 1, deep = static_cast<double>(ceil_div(stages, parts));
      const double load = (t.rows + t.cols) * 0.128 * deep / (shared > 1 ? 28 : 20);
      const double mult = e == El::F32 ? t.rows * t.cols * 64 * deep / 0.5e6 : 0;
      const double in_turn = e == El::F32 ? static_cast<double>(ceil_div(items, kCus)) : rounds * shared;
      offer(in_turn * std::max(load, mult) + 2 + (by_dma && strided ? 4.0 : 0.5) * rounds + (parts > 1 ? 4 + planes * 2 / 5e6 : 0),
            TilePlan{t.rows, t.cols, 0, tiles, 0, parts});
    }
  }
  if (!by_dma) return best;
  // Microseconds of a stage with all CUs at work (the clock falls with the power) or each
  // alone, and of a tile's begin and end; `on` tiles run on a CU at a time.  Two buffers are
  // enough where two tiles share a CU or the multiplications take long; elsewhere more keep
  // more loads on their way: 224 x 4096 x 5120 in 64 x 128 tiles takes 47 us with two, 27
  // with four, and in two parts 21 (128 x 128 24, 256 x 256 in eight parts 29).
  //
  // Weight gradients (`strided`) contract over the rows, which may be few: then a tile's begin
  // and end decide, which two tiles on a CU hide for each other.  5120 x 2048 over 224 rows takes
  // 21 us in 256 x 256, 23 in 256 x 128, 16 in 128 x 128 by twos and 20 alone; 4096 x 4096 over
  // 1000 42, 48, 43 and 53; 5120 x 17408 over 64 87, 88, 58 and 97 (75 through registers).
  static const struct { int rows, cols, bufs, on; double stage, alone, end, strided_end; } kDma[] = {
      {256, 256, 2, 1, 1.55, 1.07, 7, 13}, {256, 128, 3, 1, 0.9, 0.62, 6, 7.2}, {128, 128, 2, 2, 0.93, 0.55, 5, 4.5},
      {128, 128, 3, 1, 0.5, 0.36, 5, 4.3}, {64, 128, 2, 2, 0.69, 0.5, 4, 4}, {64, 128, 4, 1, 0.36, 0.28, 4, 4}};
  // A large tile alone on its CU, with no other row of tiles that would bring its columns into
  // the L2, waits for memory: 256 x 34816 x 5120 takes 167 us in 136 of them, 133 in
  // 128 x 128 by twos.
  const auto pace_alone = [&](const auto& t) { return t.cols == 256 && M <= 256 ? 2.0 : t.alone; };
  // Microseconds of a result's bytes beyond the first two: a CU moves about 15 KB in one.
  const double out = (out_bytes - 2) * (pair ? 0.5 : 1.0) / 15e3;
  for (const auto& t : kDma) {
    if (t.rows == 64 && strided) continue;
    // Full rounds of whole tiles; what is left over, which would leave CUs idle, in parts.
    const int64_t slots = int64_t{t.on} * kCus, tiles = ceil_div(M, t.rows) * ceil_div(width, t.cols);
    const int64_t whole = tiles / slots * slots, rest = tiles - whole;
    for (int parts = 1; parts <= kMaxParts; ++parts) {
      const double planes = static_cast<double>(rest) * parts * t.rows * t.cols * 4;
      if (parts > 1 && (rest == 0 || rest * parts > slots || planes > room || stages / parts < 4)) break;
      const double pace = rest * parts <= kCus ? pace_alone(t) : t.stage, end = strided ? t.strided_end : t.end;
      const double whole_end = end + out * t.rows * t.cols * t.on, rest_end = end + (parts > 1 ? 0 : out * t.rows * t.cols);
      offer(whole / slots * (t.stage * stages + whole_end) + (rest ? pace * ceil_div(stages, parts) + rest_end : 0) + 2 +
                (parts > 1 ? 2 + planes * 0.45e-6 : 0),
            TilePlan{t.rows, t.cols, t.bufs, tiles, whole, parts});
    }
  }
  return best;
}

// 16-byte pieces of an operand lie on 16-byte boundaries.
inline bool aligned16(const Operand& o, El e, bool kc, int64_t rows, int64_t K) {
  const int64_t unit = e == El::F32 ? 4 : e == El::BF16 ? 8 : 16;
  return o.ld % unit == 0 && (kc ? K : rows) % unit == 0 && reinterpret_cast<uintptr_t>(o.p) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(o.q) % 16 == 0;
}

template <El E, bool KA, bool KB, bool PAIR, bool ANY, class Epi>
void launch_tiles(const Product& g, const Epi& epi, const TilePlan& t, float* part, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(t.tiles * t.parts, 8) * 8);
  if (t.rows == 64) product_tile_kernel<E, KA, KB, PAIR, ANY, 64, 128><<<grid, 256, 0, s>>>(g, epi, t.parts, part);
  else product_tile_kernel<E, KA, KB, PAIR, ANY, 128, 128><<<grid, 256, 0, s>>>(g, epi, t.parts, part);
}
// float32 is bound by the matrix cores whatever the tile: small ones fill the CUs without
// parts and their sums.
template <bool KA, bool KB, bool PAIR, bool ANY, class Epi>
void launch_small_tiles(const Product& g, const Epi& epi, const TilePlan& t, float* part, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(t.tiles * t.parts, 8) * 8);
  product_tile_kernel<El::F32, KA, KB, PAIR, ANY, 64, 64><<<grid, 256, 0, s>>>(g, epi, t.parts, part);
}

// Rows whose offsets in a tile are 31-bit, and for a k-strided pair whole stages of either
// matrix.
template <El E, bool KB, bool PAIR>
bool fits_dma(const Product& g) {
  const int64_t far = int64_t{1} << 23;
  return g.a.ld * ElInfo<E>::kSize < far && g.b.ld * ElInfo<E>::kSize < far && (KB || !PAIR || g.b.half % ElInfo<E>::kStage == 0);
}

template <El E, bool KA, bool KB, bool PAIR, int BM, int BN, int BUFS, class Epi>
int launch_aligned(const Product& g, const Epi& epi, const TilePlan& t, float* part, hipStream_t s) {
  constexpr bool kPair = PAIR && KB;
  constexpr int kSlots = kCus * Aligned<E, KA, KB, PAIR, BM, BN, BUFS>::kOnCu, kGroups = BM * (kPair ? BN / 2 : BN) / 1024;
  const int64_t rest = t.tiles - t.whole;
  const unsigned grid = t.whole ? kSlots : static_cast<unsigned>(ceil_div(rest * t.parts, 8) * 8);
  product_aligned_kernel<E, KA, KB, PAIR, BM, BN, BUFS><<<grid, 256, 0, s>>>(g, epi, static_cast<int>(t.whole), t.parts, part);
  if (t.parts > 1) {
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
    product_rest_kernel<E, kPair, BM, BN><<<static_cast<unsigned>(rest * kGroups), 256, 0, s>>>(g, epi, static_cast<int>(t.whole), t.parts, part);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
}

// At most 16 rows: 16 operand columns to a workgroup while that gives two for each CU, else
// 8; below one for each CU parts of at least 16 blocks of 128 bytes.
template <El E, bool PAIR, class Epi, class Rows = AsTheyLie>
int launch_skinny(const Product& g, const Epi& epi, bool aligned, float* part, hipStream_t s, const Rows& rows = {}, size_t lds = 0) {
  const bool wide = PAIR || ceil_div(g.N, 16) >= 2 * kCus;
  const int64_t tiles = ceil_div(g.N, PAIR || !wide ? 8 : 16), blocks = ceil_div(g.K, ElInfo<E>::kStage);
  const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kCus / tiles, blocks / 16, kMaxParts})));
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(parts));
  constexpr int kThreads = kSkinnyEight * kWave;
  if (wide) {
    if (aligned) product_skinny_kernel<E, PAIR, false, 2><<<grid, kThreads, lds, s>>>(g, rows, epi, parts, part);
    else product_skinny_kernel<E, PAIR, true, 2><<<grid, kThreads, lds, s>>>(g, rows, epi, parts, part);
  } else if constexpr (!PAIR) {
    if (aligned) product_skinny_kernel<E, false, false, 1><<<grid, kThreads, lds, s>>>(g, rows, epi, parts, part);
    else product_skinny_kernel<E, false, true, 1><<<grid, kThreads, lds, s>>>(g, rows, epi, parts, part);
  }
  if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  if (parts > 1) {
    product_sum_kernel<E, PAIR><<<static_cast<unsigned>(ceil_div(g.M * part_stride(g.N) / 4, 256)), 256, 0, s>>>(g, epi, parts, part);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  }
  return MOE_OK;
}

// Up to 16 rows every workgroup of the streaming kernel reads all rows; where they and the
// weights are many that weighs more than a tile's idle rows and its parts.  Microseconds of
// the streaming kernel and of tiles: gated FFN, bf16, 16 x 4096 x 4096 32 and 34, 12 x 5120 x 8192 72
// and 63, 16 x 5120 x 17408 164 and 111; int8 9 x 5120 x 5120 12 and 14, 16 x 5120 x 5120 14 and 11,
// 4 x 5120 x 17408 25 and 25, 16 x 5120 x 17408 39 and 26.
inline bool rows_weigh(El e, int64_t M, int64_t width, int64_t K) {
  return M >= 4 && M * width * K >= (e == El::I8 ? int64_t{6} << 26 : int64_t{3} << 28);
}

// Runs a product of M, N, K >= 1; `part` holds part_bytes(pair, M, N).
template <El E, bool KA, bool KB, bool PAIR, class Epi>
int run_product(const Product& g, const Epi& epi, float* part, hipStream_t s) {
  constexpr bool kPair = PAIR && KB;
  const bool aligned = aligned16(g.a, E, KA, g.M, g.K) && aligned16(g.b, E, KB, g.N, g.K);
  bool by_dma = false;
  if constexpr (E != El::F32) by_dma = aligned && fits_dma<E, KB, PAIR>(g);
  if constexpr (KA && KB) {
    // (Strides: 32-bit offsets of the rows.)
    const bool weigh = by_dma && rows_weigh(E, g.M, kPair ? 2 * int64_t{g.N} : g.N, g.K);
    if (g.M <= kSkinnyRows && !weigh && std::max(g.a.ld, g.b.ld) < (int64_t{1} << 24)) return launch_skinny<E, PAIR>(g, epi, aligned, part, s);
  }
  const TilePlan t = plan_tiles(E, kPair, epi.bytes(), by_dma, !KA, g.M, g.N, g.K);
  if constexpr (E != El::F32) {
    if constexpr (KA) {
      if (t.bufs == 2 && t.rows == 64) return launch_aligned<E, KA, KB, PAIR, 64, 128, 2>(g, epi, t, part, s);
      if (t.bufs == 4 && t.rows == 64) return launch_aligned<E, KA, KB, PAIR, 64, 128, 4>(g, epi, t, part, s);
    }
    if (t.bufs == 2 && t.rows == 128) return launch_aligned<E, KA, KB, PAIR, 128, 128, 2>(g, epi, t, part, s);
    if (t.bufs == 3 && t.rows == 128) return launch_aligned<E, KA, KB, PAIR, 128, 128, 3>(g, epi, t, part, s);
    if (t.bufs == 3) return launch_aligned<E, KA, KB, PAIR, 256, 128, 3>(g, epi, t, part, s);
    if (t.bufs == 2) return launch_aligned<E, KA, KB, PAIR, 256, 256, 2>(g, epi, t, part, s);
  }
  if (t.cols == 64) {
    if constexpr (E == El::F32) {
      if (aligned) launch_small_tiles<KA, KB, PAIR, false>(g, epi, t, part, s);
      else launch_small_tiles<KA, KB, PAIR, true>(g, epi, t, part, s);
    }
  } else if (aligned) {
    launch_tiles<E, KA, KB, PAIR, false>(g, epi, t, part, s);
  } else {
    launch_tiles<E, KA, KB, PAIR, true>(g, epi, t, part, s);
  }
  if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  if (t.parts > 1) {
    product_sum_kernel<E, kPair><<<static_cast<unsigned>(ceil_div(g.M * part_stride(g.N) / 4, 256)), 256, 0, s>>>(g, epi, t.parts, part);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe
