// Dense matrix product with its epilogue: y = act(x W^T + bias) + residual.
//
// Sums run in float32 over the whole contraction; bias, activation and residual are
// applied to the float32 sum, which is rounded once, to y's type.  Four kernels:
//
//   linear_skinny_kernel  at most 16 rows of x: streams W, see skinny.h;
//   linear_tile_kernel    more rows: tiles through LDS, any alignment;
//   linear_wide_kernel    enough rows and columns to fill the GPU with 256 x 256 tiles
//                         (aligned bf16): the matrix cores' rate;
//   linear_any_kernel     strides too large for the others' offsets.
//
// When their tiles do not fill the GPU the first two cut the contraction into parts,
// whose sums a second launch adds in order and finishes.
#include <algorithm>

#include "moe_mi355x.h"
#include "dma.h"
#include "skinny.h"

namespace moe {
namespace {

struct LinearArgs {
  const void *x, *w, *bias, *residual;
  void* y;
  int64_t ldx, ldw, ldr, ldy;    // elements
  int M, N, K;
  int act;
};

// Floats between rows of a plane of partial sums.
__host__ __device__ inline int64_t part_stride(int64_t N) { return (N + 3) / 4 * 4; }

// ---------------------------------------------------------------- epilogue

// v / (1 + e^-u): silu with u = v, and with u = 2 sqrt(2/pi) (v + 0.044715 v^3) the tanh
// form of gelu, as (1 + tanh(u/2)) / 2 = 1 / (1 + e^-u); e^-u = inf gives 0.  QUICK: the
// hardware's exponential and reciprocal, good to 2^-22 (1 + |u|), for results that are
// rounded to bf16.
template <bool QUICK>
__device__ __forceinline__ float gated(float v, float u) {
  if constexpr (QUICK) return v * __builtin_amdgcn_rcpf(1.0f + __expf(-u));
  else return v / (1.0f + expf(-u));
}

template <bool QUICK, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = v[c] < 0.0f ? 0.0f : v[c];             // NaN stays NaN
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = 0.5f * v[c] * (1.0f + erff(v[c] * 0.70710678f));
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = gated<QUICK>(v[c], 1.59576912f * (v[c] + 0.044715f * v[c] * v[c] * v[c]));
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int c = 0; c < N; ++c) v[c] = gated<QUICK>(v[c], v[c]);
      break;
    default:
      break;
  }
}

template <bool F32>
__device__ __forceinline__ float elem(const void* p, size_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// One output element from its float32 sum.
template <bool F32, bool OUT32>
__device__ __forceinline__ void finish(const LinearArgs& a, int m, int n, float v) {
  float t[1] = {a.bias ? v + elem<F32>(a.bias, n) : v};
  activate<!OUT32>(t, a.act);
  v = t[0];
  if (a.residual) v += elem<OUT32>(a.residual, static_cast<size_t>(m) * a.ldr + n);
  const size_t o = static_cast<size_t>(m) * a.ldy + n;
  if constexpr (OUT32) static_cast<float*>(a.y)[o] = v;
  else static_cast<uint16_t*>(a.y)[o] = f32_to_bf16_bits(v);
}

// Four neighbouring elements; these accesses need only the elements' alignment.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32>
__device__ __forceinline__ f32x4 load4(const void* p, size_t i) {
  f32x4 v;
  if constexpr (F32) {
    const f32x4_any q = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = q[c];
  } else {
    const u16x4_any q = *reinterpret_cast<const u16x4_any*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = bf16_bits_to_f32(q[c]);
  }
  return v;
}
template <bool F32>
__device__ __forceinline__ void store4(void* p, size_t i, const float* v) {
  if constexpr (F32) {
    *reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + i) = f32x4_any{v[0], v[1], v[2], v[3]};
  } else {
    u16x4_any o;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = f32_to_bf16_bits(v[c]);
    *reinterpret_cast<u16x4_any*>(static_cast<uint16_t*>(p) + i) = o;
  }
}

// D rows of four neighbouring columns from n on (rows m[d], of which those past the end
// are left out).  The residual's loads are in flight together.
template <bool F32, bool OUT32, int D>
__device__ __forceinline__ void finish_quads(const LinearArgs& a, const int (&m)[D], int n, const f32x4 (&s)[D]) {
  if (n + 4 > a.N) {
#pragma unroll 1
    for (int d = 0; d < D; ++d)
      for (int c = 0; c < 4; ++c)
        if (m[d] < a.M && n + c < a.N) finish<F32, OUT32>(a, m[d], n + c, s[d][c]);
    return;
  }
  f32x4 res[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    res[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.residual && m[d] < a.M) res[d] = load4<OUT32>(a.residual, static_cast<size_t>(m[d]) * a.ldr + n);
  }
  f32x4 bias = {0.f, 0.f, 0.f, 0.f};
  if (a.bias) bias = load4<F32>(a.bias, n);
  float v[4 * D];
#pragma unroll
  for (int d = 0; d < D; ++d)
#pragma unroll
    for (int c = 0; c < 4; ++c) v[4 * d + c] = s[d][c] + bias[c];
  activate<!OUT32>(v, a.act);
#pragma unroll
  for (int d = 0; d < D; ++d) {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[4 * d + c] += res[d][c];
    if (m[d] < a.M) store4<OUT32>(a.y, static_cast<size_t>(m[d]) * a.ldy + n, v + 4 * d);
  }
}

// ROWS x BN sums in LDS, rows `stride` floats apart, as y or as part p's sums: row_of(R)
// is the row of y behind row R.  Whole row segments, four columns to a thread.
template <bool F32, bool OUT32, int BN, int ROWS, int THREADS, class RowOf>
__device__ __forceinline__ void finish_rows(const LinearArgs& a, const float* stg, int stride, int n0, int parts, int p,
                                            float* part, RowOf row_of) {
  constexpr int kLanes = BN / 4, kIter = ROWS * kLanes / THREADS, D = 4;
  static_assert(THREADS % kLanes == 0 && kIter % D == 0, "a thread keeps its columns");
  const int tid = threadIdx.x, c = 4 * (tid % kLanes), n = n0 + c;
  if (n >= a.N) return;
#pragma unroll 1
  for (int k = 0; k < kIter; k += D) {
    int m[D];
    f32x4 s[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int R = (tid + (k + d) * THREADS) / kLanes;
      m[d] = row_of(R);
      s[d] = *reinterpret_cast<const f32x4*>(stg + R * stride + c);
    }
    if (parts > 1) {
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (m[d] < a.M)
          *reinterpret_cast<f32x4*>(part + (static_cast<size_t>(p) * a.M + m[d]) * part_stride(a.N) + n) = s[d];
    } else {
      finish_quads<F32, OUT32, D>(a, m, n, s);
    }
  }
}

// Eight bf16 of a row, of which it holds the first n more (ANY: 2-byte aligned).
template <bool ANY>
__device__ __forceinline__ uint4 ld8_bf16(const uint16_t* p, int n) {
  if (n >= 8) {
    if constexpr (ANY) {
      typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
      const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p);
      return uint4{v.x, v.y, v.z, v.w};
    }
    return ld16(p);
  }
  uint32_t v[4] = {0, 0, 0, 0};
  if constexpr (ANY) {               // aligned rows are multiples of 8 long
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) v[k >> 1] |= static_cast<uint32_t>(p[k]) << (16 * (k & 1));
  }
  return uint4{v[0], v[1], v[2], v[3]};
}
// 16 bytes of a row from element k on, zeros past its end.
template <bool F32, bool ANY>
__device__ __forceinline__ uint4 ld_piece(const void* row, int k, int kdim) {
  if constexpr (F32) return ld_f32x4(static_cast<const uint8_t*>(row) + 4 * static_cast<size_t>(k), kdim - k, !ANY);
  else return ld8_bf16<ANY>(static_cast<const uint16_t*>(row) + k, kdim - k);
}

// ---------------------------------------------------------------- at most 16 rows
//
// A workgroup of eight waves computes 8 SETS columns over one part of the contraction,
// an eighth for each wave.  Short batches and many waves (three workgroups on a CU with
// 8 columns, two with 16): four waves with batches three times as long took twice the
// time on 1 x 5120 x 5120, which now takes 13.6 us (52 MB: 3.9 TB/s; bound by the start
// and the drain of one short grid); 7 x 5120 x 17408 takes 40.6 (178 MB: 4.4 TB/s; the
// loads of x are about 15 % of it, the rest is the memory's).  With 8 columns the weights of a block are one register,
// and the two halves of the block are multiplied apart (each over all 16 columns of
// the MFMA, of which 8 are its own).
constexpr int kSkinnyWaves = 8;

template <bool F32, bool OUT32, bool ANY, int SETS>
__global__ void __launch_bounds__(kSkinnyWaves * kWave, SETS == 1 ? 6 : 4) linear_skinny_kernel(LinearArgs a, int parts, float* part) {
  constexpr int FMT = F32 ? kDtypeF32 : kDtypeBf16;
  constexpr int kBlk = SkinnyFmt<FMT>::kBlk, kPiece = F32 ? 4 : 8, kSize = F32 ? 4 : 2;
  constexpr int D = SETS == 1 ? 4 : 5;
  __shared__ f32x4 red[kSkinnyWaves][kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (8 * SETS), p = blockIdx.y;
  const int nb = static_cast<int>(ceil_div(a.K, kBlk));
  const int b0 = static_cast<int>(static_cast<int64_t>(p) * nb / parts), b1 = static_cast<int>(static_cast<int64_t>(p + 1) * nb / parts);
  const int lo = b0 + wave * (b1 - b0) / kSkinnyWaves, hi = b0 + (wave + 1) * (b1 - b0) / kSkinnyWaves;
  // Rows within the first one's 4 GiB (the host checks the strides).
  const uint8_t* wbase = static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * a.ldw * kSize;
  const uint8_t* xbase = static_cast<const uint8_t*>(a.x);
  uint32_t woff[SETS];
#pragma unroll
  for (int h = 0; h < SETS; ++h)
    woff[h] = static_cast<uint32_t>(min(8 * h + (lane & 7), a.N - 1 - n0)) * static_cast<uint32_t>(a.ldw) * kSize +
              16 * lane_piece(lane);
  const uint32_t xoff = static_cast<uint32_t>(min(r, a.M - 1)) * static_cast<uint32_t>(a.ldx) * kSize + 16 * g;
  const bool live = r < a.M;
  const bool tail = a.K % kBlk != 0;

  struct Blk {
    uint4 w[SETS], x[2];
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  int at = lo;
  batches<D, Blk>(
      hi - lo,
      [&](Blk& k) __attribute__((always_inline)) {
        const uint8_t* wb = wbase + static_cast<size_t>(at) * kBlkBytes;
        const uint8_t* xb = xbase + static_cast<size_t>(at) * kBlkBytes;
        // Elements of the row from this block on; only the last block can be cut.
        const int left = a.K - at * kBlk;
        k.x[0] = k.x[1] = uint4{0, 0, 0, 0};
        if (!ANY && !tail) {
#pragma unroll
          for (int h = 0; h < SETS; ++h) k.w[h] = ld16_stream(wb + woff[h]);
          if (live) {
            k.x[0] = ld16(xb + xoff);
            k.x[1] = ld16(xb + xoff + 64);
          }
        } else {
#pragma unroll
          for (int h = 0; h < SETS; ++h) k.w[h] = ld_piece<F32, ANY>(wb + woff[h], 0, left - kPiece * lane_piece(lane));
          if (live) {
            k.x[0] = ld_piece<F32, ANY>(xb + xoff, 0, left - kPiece * g);
            k.x[1] = ld_piece<F32, ANY>(xb + xoff + 64, 0, left - kPiece * (g + 4));
          }
        }
        ++at;
      },
      [&](Blk& k) __attribute__((always_inline)) {
        if constexpr (SETS == 2) {
          WBlk<FMT> w;
          w.v[0] = k.w[0];
          w.v[1] = k.w[1];
          XBlk<FMT> x[1];
          x[0].v[0][0] = k.x[0];
          x[0].v[1][0] = k.x[1];
          acc[0] = mma_planes<FMT, 1>(x, w, lane, acc[0]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (F32) {
              acc[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k.x[h].x), __uint_as_float(k.w[0].x), acc[h], 0, 0, 0);
              acc[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k.x[h].y), __uint_as_float(k.w[0].y), acc[h], 0, 0, 0);
              acc[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k.x[h].z), __uint_as_float(k.w[0].z), acc[h], 0, 0, 0);
              acc[h] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k.x[h].w), __uint_as_float(k.w[0].w), acc[h], 0, 0, 0);
            } else {
              acc[h] = mfma_bf16_16x16x32(k.x[h], k.w[0], acc[h]);
            }
          }
        }
      },
      [] {});
  f32x4 s = acc[0];
  if constexpr (SETS == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = (lane & 8) ? acc[1][i] : acc[0][i];
      s[i] = v + __shfl_xor(v, 8, kWave);
    }
  }
  red[wave][lane] = s;
  __syncthreads();
  // Wave w < 4 finishes elements i = w: rows 4 g + w.
  if (wave >= 4) return;
  float v = red[0][lane][wave];
#pragma unroll
  for (int o = 1; o < kSkinnyWaves; ++o) v += red[o][lane][wave];
  const int m = 4 * g + wave, n = n0 + r;
  if (m < a.M && n < a.N && r < 8 * SETS) {
    if (parts > 1) part[(static_cast<size_t>(p) * a.M + m) * part_stride(a.N) + n] = v;
    else finish<F32, OUT32>(a, m, n, v);
  }
}

// ---------------------------------------------------------------- LDS tiles
//
// BM x BN outputs per workgroup of 2 x 2 waves, from 32x32 MFMAs.  A stage is 128 bytes
// of each row (64 bf16 or 32 f32), double-buffered in LDS; its loads go to registers
// two stages ahead, which takes any alignment and fills the row ends with zeros.  Rows
// are stored unpadded with their 16-byte pieces permuted by (row / 2) mod 8, so that a
// fragment read touches each bank group once per 16 rows.
// Bound by the bytes that a CU takes in, about 28 KB in a microsecond: 1001 x 1537 x 2049
// bf16 with odd row strides 27 us and 9 for its parts' sum.  Small products are bound by
// the loads' latency before the first multiplication and by the results' way out:
// 333 x 1023 x 515 f32 in 8 parts of 4 stages takes 17 us and 4 for the sum, a product
// of one stage 15; on 16-byte boundaries, one load in place of four, 12 and 4.
// The results leave through LDS as row segments with four residual loads in flight; with
// one element at a time 715 x 64 x 15104 took 72 us instead of 28.
// Tiles that share rows of W are neighbours on one XCD (workgroup b runs on XCD b % 8).
__device__ __forceinline__ int xcd_tile(int b, int total) {
  const int per = (total + 7) / 8;
  return b / 8 < per && (b % 8) * per + b / 8 < total ? (b % 8) * per + b / 8 : -1;
}

template <bool F32, bool OUT32, bool ANY, int BM, int BN>
__global__ void __launch_bounds__(256, 2) linear_tile_kernel(LinearArgs a, int parts, float* part) {
  constexpr int kElems = F32 ? 32 : 64, kPiece = F32 ? 4 : 8, kSize = F32 ? 4 : 2;
  constexpr int RA = BM / 32, RB = BN / 32, NI = BM / 64, NJ = BN / 64;
  constexpr int kStage = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hi = lane >> 5;
  const int mt = static_cast<int>(ceil_div(a.M, BM)), nt = static_cast<int>(ceil_div(a.N, BN));
  const int item = xcd_tile(blockIdx.x, mt * nt * parts);
  if (item < 0) return;
  const int p = item % parts, m0 = (item / parts) % mt * BM, n0 = (item / parts) / mt * BN;
  const int stages = static_cast<int>(ceil_div(a.K, kElems));
  const int s0 = static_cast<int>(static_cast<int64_t>(p) * stages / parts), s1 = static_cast<int>(static_cast<int64_t>(p + 1) * stages / parts);

  // Thread t loads piece t % 8 of rows t / 8 + 32 q; rows past the end repeat the last.
  const int row = tid >> 3, piece = tid & 7;
  const uint8_t* xbase = static_cast<const uint8_t*>(a.x) + static_cast<size_t>(m0) * a.ldx * kSize;
  const uint8_t* wbase = static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * a.ldw * kSize;
  uint32_t xoff[RA], woff[RB];
#pragma unroll
  for (int q = 0; q < RA; ++q)
    xoff[q] = static_cast<uint32_t>(min(row + 32 * q, a.M - 1 - m0)) * static_cast<uint32_t>(a.ldx) * kSize + 16 * piece;
#pragma unroll
  for (int q = 0; q < RB; ++q)
    woff[q] = static_cast<uint32_t>(min(row + 32 * q, a.N - 1 - n0)) * static_cast<uint32_t>(a.ldw) * kSize + 16 * piece;
  struct Regs {
    uint4 x[RA], w[RB];
  };
  auto load = [&](Regs& R, int s) __attribute__((always_inline)) {
    const int st = min(s, s1 - 1), left = a.K - st * kElems - piece * kPiece;
    const uint8_t* xb = xbase + static_cast<size_t>(st) * 128;
    const uint8_t* wb = wbase + static_cast<size_t>(st) * 128;
#pragma unroll
    for (int q = 0; q < RA; ++q) R.x[q] = ld_piece<F32, ANY>(xb + xoff[q], 0, left);
#pragma unroll
    for (int q = 0; q < RB; ++q) R.w[q] = ld_piece<F32, ANY>(wb + woff[q], 0, left);
  };
  const uint32_t lds = static_cast<uint32_t>(row * 128 + ((piece ^ ((row >> 1) & 7)) * 16));
  auto store = [&](const Regs& R, int buf) __attribute__((always_inline)) {
    uint8_t* d = smem + buf * kStage + lds;
#pragma unroll
    for (int q = 0; q < RA; ++q) *reinterpret_cast<uint4*>(d + 32 * q * 128) = R.x[q];
#pragma unroll
    for (int q = 0; q < RB; ++q) *reinterpret_cast<uint4*>(d + BM * 128 + 32 * q * 128) = R.w[q];
  };
  f32x16 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  const uint32_t swz = static_cast<uint32_t>(hi ^ ((r32 >> 1) & 7));
  auto compute = [&](int buf) __attribute__((always_inline)) {
    const uint8_t* As = smem + buf * kStage + (wm * (BM / 2) + r32) * 128;
    const uint8_t* Bs = smem + buf * kStage + (BM + wn * (BN / 2) + r32) * 128;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t pc = ((2 * kk) ^ swz) * 16;
      uint4 xf[NI], wf[NJ];
#pragma unroll
      for (int i = 0; i < NI; ++i) xf[i] = *reinterpret_cast<const uint4*>(As + i * 32 * 128 + pc);
#pragma unroll
      for (int j = 0; j < NJ; ++j) wf[j] = *reinterpret_cast<const uint4*>(Bs + j * 32 * 128 + pc);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if constexpr (F32) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(xf[i].x), __uint_as_float(wf[j].x), acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(xf[i].y), __uint_as_float(wf[j].y), acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(xf[i].z), __uint_as_float(wf[j].z), acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(xf[i].w), __uint_as_float(wf[j].w), acc[i][j], 0, 0, 0);
          } else {
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, xf[i]), __builtin_bit_cast(bf16x8, wf[j]), acc[i][j], 0, 0, 0);
          }
        }
    }
  };

  // Iteration s: barrier; write stage s + 1 from registers, start loading s + 3 into
  // them (past the end the last stage again), multiply stage s.
  Regs R0, R1;
  load(R0, s0);
  load(R1, s0 + 1);
  store(R0, 0);
  load(R0, s0 + 2);
  for (int s = s0; s < s1; s += 2) {
    __syncthreads();
    store(R1, 1);
    load(R1, s + 3);
    compute(0);
    if (s + 1 == s1) break;
    __syncthreads();
    store(R0, 0);
    load(R0, s + 4);
    compute(1);
  }

  // Out through LDS, NI rounds of 32 rows of each wave row, rows padded by 8 floats.
  // Lane l, element v: row 8 (v / 4) + 4 (l / 32) + v % 4, column l % 32 of a block.
  constexpr int kStride = BN + 8;
  static_assert(64 * kStride * 4 <= 2 * kStage, "a round fits the stage buffers");
  float* stg = reinterpret_cast<float*>(smem);
  __syncthreads();                   // every wave is done reading the stage buffers
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int v = 0; v < 16; ++v)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        stg[(wm * 32 + 8 * (v >> 2) + 4 * hi + (v & 3)) * kStride + wn * (BN / 2) + 32 * j + r32] = acc[i][j][v];
    __syncthreads();
    finish_rows<F32, OUT32, BN, 64, 256>(a, stg, kStride, n0, parts, p, part, [&](int R) {
      return m0 + (R / 32) * (BM / 2) + 32 * i + R % 32;
    });
    __syncthreads();
  }
}

// ---------------------------------------------------------------- 256-row tiles
//
// 256 x BN outputs per workgroup of 8 waves, two per SIMD, so that one wave's fragment
// reads and waits overlap the other's MFMAs.  A wave computes 128 x 64 (BN = 256) or
// 64 x 64 (BN = 128) outputs in blocks of 32x32x16 MFMAs.
// A stage is 64 elements, 128 bytes of each row, double-buffered in LDS: the rows of x
// go there by DMA one stage ahead, the rows of W through registers two stages ahead,
// which keeps two stages of the HBM stream in flight within the LDS.  Tiles are walked
// in bands of 8 row blocks, so that the 32 tiles that run on an XCD at a time share 8
// row blocks and 4 column blocks in its L2.
// 8192 x 7168 x 4096: 418 to 439 us in a row of calls, 1.10 to 1.15 PFLOP/s (the library's product
// alone 371 us; under the profiler 442 to 553 us, the median 471), bound by the matrix
// cores; 224 x 5120 x 5120 in 240 items of 6 parts: 20 to 24 us, bound by the bytes that a
// CU takes in (36 KB in a microsecond), and 8 for its parts' sum (the library's product
// alone 47).
constexpr int kWideRows = 256, kWideThreads = 512;
constexpr int kWideRow = 128;
constexpr int kWideBand = 8;

template <bool OUT32, int BN>
__global__ void __launch_bounds__(kWideThreads) linear_wide_kernel(LinearArgs a, int parts, float* part) {
  constexpr int kStage = (kWideRows + BN) * kWideRow;
  constexpr int WN = BN / 64, WM = 8 / WN, NI = kWideRows / WM / 32, NB = BN / 64;   // NB: W pieces per thread
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, r32 = lane & 31, hi = lane >> 5;
  const int mt = static_cast<int>(ceil_div(a.M, kWideRows)), nt = static_cast<int>(ceil_div(a.N, BN));
  const uint32_t xrow = static_cast<uint32_t>(a.ldx) * 2, wrow = static_cast<uint32_t>(a.ldw) * 2;
  const int pairs = a.K / 128;               // of stages

  // DMA instruction q of this wave covers tile rows 8 (4 wave + q) + lane / 8; LDS piece
  // lane % 8 holds global piece (lane % 8) ^ ((row / 2) mod 8).
  const int drow = lane >> 3;
  uint32_t dpiece[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) dpiece[h] = static_cast<uint32_t>(((lane & 7) ^ ((4 * h + (drow >> 1)) & 7)) * 16);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(smem));
  const uint32_t fswz = static_cast<uint32_t>(hi ^ ((r32 >> 1) & 7));
  const uint32_t bldsoff = static_cast<uint32_t>((tid >> 3) * kWideRow + (((tid & 7) ^ ((tid >> 4) & 7)) * 16));

  const XcdWalk walk(mt * nt * parts);
  for (int item = walk.tile; item < walk.end; item += walk.step) {
    const int tile = item / parts, p = item - tile * parts;
    // Stages [k0, nk), an even number of them (the host sends contractions of whole pairs).
    const int k0 = 2 * (p * pairs / parts), nk = 2 * ((p + 1) * pairs / parts);
    const int band = tile / (kWideBand * nt), in_band = tile - band * kWideBand * nt;
    const int bm = min(kWideBand, mt - band * kWideBand);
    const int m0 = (band * kWideBand + in_band % bm) * kWideRows, n0 = in_band / bm * BN;
    // Rows past the end repeat the last one; their sums are not stored.  The descriptors
    // cover the tile's rows, the host's bound on the strides keeps them below 4 GiB.
    const int xr = min(kWideRows, a.M - m0) - 1, wr = min(BN, a.N - n0) - 1;
    const i32x4_t ra = dma_rsrc(static_cast<const uint8_t*>(a.x) + static_cast<size_t>(m0) * xrow,
                                static_cast<uint32_t>(xr) * xrow + static_cast<uint32_t>(a.K) * 2);
    const __amdgpu_buffer_rsrc_t rb = buf_rsrc(static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * wrow,
                                               static_cast<uint32_t>(wr) * wrow + static_cast<uint32_t>(a.K) * 2);
    uint32_t aoff[4], boff[NB];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      aoff[q] = static_cast<uint32_t>(min(8 * (4 * wave + q) + drow, xr)) * xrow + dpiece[q & 1];
#pragma unroll
    for (int q = 0; q < NB; ++q)
      boff[q] = static_cast<uint32_t>(min((tid >> 3) + 64 * q, wr)) * wrow + (tid & 7) * 16;
    auto issue_a = [&](int ks) __attribute__((always_inline)) {
      dma4_rows(ra, aoff, static_cast<uint32_t>(ks) * kWideRow,
                lds0 + static_cast<uint32_t>(ks & 1) * kStage + 4 * wave * 1024);
    };
    struct BRegs {
      uint4 v[NB];
    };
    auto load_b = [&](BRegs& R, int ks) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < NB; ++q) R.v[q] = buf_ld16(rb, boff[q], static_cast<uint32_t>(ks) * kWideRow);
    };
    auto store_b = [&](const BRegs& R, int ks) __attribute__((always_inline)) {
      uint8_t* dst = smem + (ks & 1) * kStage + kWideRows * kWideRow + bldsoff;
#pragma unroll
      for (int q = 0; q < NB; ++q) *reinterpret_cast<uint4*>(dst + 64 * q * kWideRow) = R.v[q];
    };
    f32x16 acc[NI][2];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    auto compute = [&](int ks) __attribute__((always_inline)) {
      const uint8_t* base = smem + (ks & 1) * kStage;
      const uint8_t* As = base + (wm * 32 * NI + r32) * kWideRow;
      const uint8_t* Bs = base + (kWideRows + wn * 64 + r32) * kWideRow;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t piece = ((2 * kk) ^ fswz) * 16;
        uint4 af[NI], bf[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) bf[j] = *reinterpret_cast<const uint4*>(Bs + 32 * j * kWideRow + piece);
#pragma unroll
        for (int i = 0; i < NI; ++i) af[i] = *reinterpret_cast<const uint4*>(As + 32 * i * kWideRow + piece);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16_32x32x16(af[i], bf[j], acc[i][j]);
      }
    };
    // Iteration ks: wait for x(ks); barrier; write W(ks + 1) from registers and start
    // x(ks + 1) into the other buffer; refill those registers with W(ks + 3); multiply
    // stage ks.  Past the end the last stage of W is read again, so that every iteration
    // has the same number of loads in flight.
    BRegs R0, R1;
    load_b(R0, k0);
    load_b(R1, k0 + 1);
    __syncthreads();                 // the previous tile is done with both buffers
    store_b(R0, k0);
    issue_a(k0);
    load_b(R0, min(k0 + 2, nk - 1));
    for (int ks = k0; ks < nk; ks += 2) {
      wait_vm<NB>();
      __syncthreads();
      store_b(R1, ks + 1);
      issue_a(ks + 1);
      load_b(R1, min(ks + 3, nk - 1));
      compute(ks);
      wait_vm<NB>();
      __syncthreads();
      if (ks + 2 < nk) {
        store_b(R0, ks + 2);
        issue_a(ks + 2);
      }
      load_b(R0, min(ks + 4, nk - 1));
      compute(ks + 1);
    }
    wait_vm<0>();                    // no load may still be writing registers or LDS
    __syncthreads();                 // every wave is done reading the stage buffers

    // Out through LDS, so that bias, residual and y (or the part's sums) are taken in
    // whole row segments, four columns to a lane.  NI rounds of 32 rows of each wave row;
    // rows padded by 8 floats.
    constexpr int kStride = BN + 8;
    static_assert(32 * WM * kStride * 4 <= 2 * kStage, "a round fits the stage buffers");
    float* stg = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int v = 0; v < 16; ++v)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          stg[(wm * 32 + 8 * (v >> 2) + 4 * hi + (v & 3)) * kStride + wn * 64 + 32 * j + r32] = acc[i][j][v];
      __syncthreads();
      finish_rows<false, OUT32, BN, 32 * WM, kWideThreads>(a, stg, kStride, n0, parts, p, part, [&](int R) {
        return m0 + (R / 32 * NI + i) * 32 + R % 32;
      });
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- parts added up

// A thread adds up four neighbouring sums, all parts' loads in flight together as far as
// kPartsAhead goes.  Rows of a plane are padded to multiples of four.
constexpr int kPartsAhead = 8;

template <bool F32, bool OUT32>
__global__ void __launch_bounds__(256) linear_finish_kernel(LinearArgs a, int parts, const float* part) {
  const int quads = static_cast<int>(part_stride(a.N) / 4);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.M) * quads) return;
  const int64_t plane = static_cast<int64_t>(a.M) * quads;
  const f32x4* v = reinterpret_cast<const f32x4*>(part) + i;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < parts; p += kPartsAhead) {
    f32x4 b[kPartsAhead];
#pragma unroll
    for (int k = 0; k < kPartsAhead; ++k)
      if (p + k < parts) b[k] = v[plane * (p + k)];
#pragma unroll
    for (int k = 0; k < kPartsAhead; ++k)
      if (p + k < parts)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[c] += b[k][c];
  }
  const int m[1] = {static_cast<int>(i / quads)};
  const f32x4 t[1] = {s};
  finish_quads<F32, OUT32, 1>(a, m, 4 * static_cast<int>(i - static_cast<int64_t>(m[0]) * quads), t);
}

// ---------------------------------------------------------------- any stride
//
// 64 x 64 outputs per workgroup of 4 waves, stages of 32 contraction elements read
// element by element.
constexpr int kAnyTile = 64, kAnyK = 32;

template <bool F32, bool OUT32>
__global__ void __launch_bounds__(256) linear_any_kernel(LinearArgs a) {
  using E = std::conditional_t<F32, float, uint16_t>;
  constexpr int kPad = F32 ? 4 : 8;
  __shared__ __attribute__((aligned(16))) E xs[kAnyTile][kAnyK + kPad], wsm[kAnyTile][kAnyK + kPad];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kAnyTile, n0 = static_cast<int64_t>(blockIdx.x) * kAnyTile;
  const E* x = static_cast<const E*>(a.x);
  const E* w = static_cast<const E*>(a.w);
  f32x4 acc[4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kAnyK) {
    for (int i = tid; i < kAnyTile * kAnyK; i += 256) {
      const int row = i / kAnyK, k = k0 + i % kAnyK;
      xs[row][i % kAnyK] = (m0 + row < a.M && k < a.K) ? x[(m0 + row) * a.ldx + k] : E(0);
      wsm[row][i % kAnyK] = (n0 + row < a.N && k < a.K) ? w[(n0 + row) * a.ldw + k] : E(0);
    }
    __syncthreads();
    if constexpr (F32) {
#pragma unroll
      for (int k = 0; k < kAnyK; k += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[16 * wave + r][k + g], wsm[16 * j + r][k + g], acc[j], 0, 0, 0);
    } else {
      const uint4 xf = *reinterpret_cast<const uint4*>(&xs[16 * wave + r][8 * g]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j] = mfma_bf16_16x16x32(xf, *reinterpret_cast<const uint4*>(&wsm[16 * j + r][8 * g]), acc[j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 16 * wave + 4 * g + i, n = n0 + 16 * j + r;
      if (m < a.M && n < a.N) finish<F32, OUT32>(a, static_cast<int>(m), static_cast<int>(n), acc[j][i]);
    }
}

// ---------------------------------------------------------------- host

int check_linear(const moe_linear_config* c, int32_t rows) {
  if (!c) return MOE_ERR_NULL_PTR;
  const bool f32 = c->in_dtype == MOE_DTYPE_F32 && c->out_dtype == MOE_DTYPE_F32;
  const bool bf16 = c->in_dtype == MOE_DTYPE_BF16 &&
                    (c->out_dtype == MOE_DTYPE_BF16 || c->out_dtype == MOE_DTYPE_F32);
  if (!f32 && !bf16) return MOE_ERR_BAD_DTYPE;
  if (c->in_features <= 0 || c->out_features <= 0 || rows < 0) return MOE_ERR_BAD_SHAPE;
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_SILU) return MOE_ERR_BAD_SHAPE;
  // Grid and index arithmetic inside the kernels.
  if (c->in_features > MOE_LINEAR_MAX_FEATURES || c->out_features > MOE_LINEAR_MAX_FEATURES ||
      rows > MOE_LINEAR_MAX_ROWS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// How a product runs: which tiles, and in how many parts of the contraction.
struct LinearPlan {
  int rows, cols;    // of a tile (rows 16: the skinny kernel; 256: the 256-row tiles)
  int64_t tiles;
  int parts;
};
constexpr int kCus = 256;
constexpr int kMaxParts = 16;
// Most bytes of partial sums, which linear_plan keeps to: those of two 128 x 128 tiles or
// one 256 x 128 tile on each CU.
constexpr size_t kMaxPartBytes = size_t{2} * kCus * 128 * 128 * sizeof(float);

// The cheapest plan by an estimate in microseconds.  A CU takes about 36 KB of operands
// in a microsecond in the 256-row kernel and 28 KB in the other (measured; what limits
// both in bf16), multiplies about 0.5 MFLOP f32, and partial sums cross at 5 TB/s twice.
// That prices the second launch at about twice its time: 15 us for 224 x 5120 x 5120 in 6
// parts and 14 for 1001 x 1537 x 2049 in 3, which take 8 and 9.
LinearPlan linear_plan(const moe_linear_config& c, int64_t M, bool wide) {
  const int64_t N = c.out_features, K = c.in_features;
  const bool f32 = c.in_dtype == MOE_DTYPE_F32;
  LinearPlan p{};
  if (M <= kSkinnyRows) {
    // 16 columns while that gives two workgroups for each CU, else 8; below one workgroup
    // for each CU parts of at least 16 blocks.
    p.rows = kSkinnyRows;
    p.cols = ceil_div(N, 16) >= 2 * kCus ? 16 : 8;
    p.tiles = ceil_div(N, p.cols);
    const int64_t blocks = ceil_div(K * (f32 ? 4 : 2), kBlkBytes);
    p.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kCus / p.tiles, blocks / 16, kMaxParts})));
    return p;
  }
  static const struct { int rows, cols, on_cu; } kTiles[] = {{64, 128, 2}, {128, 128, 2}, {256, 128, 1}, {256, 256, 1}};
  const int64_t stages = ceil_div(K * (f32 ? 4 : 2), 128);
  double best = 0;
  for (const auto& t : kTiles) {
    if (t.rows == kWideRows && !wide) continue;
    const int64_t tiles = ceil_div(M, t.rows) * ceil_div(N, t.cols);
    const int64_t slots = static_cast<int64_t>(t.on_cu) * kCus;
    for (int parts = 1; parts <= kMaxParts; ++parts) {
      // f32 tiles are bound by the matrix cores, so a CU may also take a few parts in turn:
      // 1529 x 4224 x 1920 took 307 us in 180 tiles of 128 x 128 (76 CUs idle), 239 in 720
      // half tiles of 64 x 128 (the library's product with the epilogue apart: 205).
      const int64_t most = f32 ? int64_t{2} * slots : slots;
      if (parts > 1 && (tiles * parts > most || parts * M * part_stride(N) * 4 > static_cast<int64_t>(kMaxPartBytes) ||
                        stages / parts < 4 || t.cols == 256))
        break;
      const int64_t items = tiles * parts, rounds = ceil_div(items, slots);
      const double shared = items > kCus ? t.on_cu : 1;             // tiles that share a CU
      const double deep = static_cast<double>(ceil_div(stages, parts));
      const double load = (t.rows + t.cols) * 0.128 * deep / (t.rows == kWideRows ? 36 : shared > 1 ? 28 : 20);
      const double mult = f32 ? t.rows * t.cols * 64 * deep / 0.5e6 : 0;
      const double in_turn = f32 ? static_cast<double>(ceil_div(items, kCus)) : rounds * shared;
      const double us = in_turn * std::max(load, mult) + 2 + 0.5 * rounds +
                        (parts > 1 ? 4 + parts * static_cast<double>(M) * N * 8 / 5e6 : 0);
      if (p.tiles == 0 || us < best) {
        best = us;
        p = LinearPlan{t.rows, t.cols, tiles, parts};
      }
    }
  }
  return p;
}

// Bytes of partial sums of any call of at most M rows.
size_t linear_workspace(const moe_linear_config& c, int64_t M) {
  const double want = static_cast<double>(kMaxParts) * M * part_stride(c.out_features) * sizeof(float);
  return want < static_cast<double>(kMaxPartBytes) ? std::max<size_t>(static_cast<size_t>(want), 256) : kMaxPartBytes;
}

bool off(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == MOE_DTYPE_F32 ? 4 : 2) != 0; }

template <bool F32, bool OUT32, bool ANY>
void linear_launch(const LinearArgs& a, const LinearPlan& p, float* part, hipStream_t s) {
  if (p.rows == kSkinnyRows) {
    const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.parts));
    if (p.cols == 16) linear_skinny_kernel<F32, OUT32, ANY, 2><<<grid, kSkinnyWaves * kWave, 0, s>>>(a, p.parts, part);
    else linear_skinny_kernel<F32, OUT32, ANY, 1><<<grid, kSkinnyWaves * kWave, 0, s>>>(a, p.parts, part);
  } else {
    const unsigned grid = static_cast<unsigned>(ceil_div(p.tiles * p.parts, 8) * 8);
    if (p.rows == 64) linear_tile_kernel<F32, OUT32, ANY, 64, 128><<<grid, 256, 0, s>>>(a, p.parts, part);
    else linear_tile_kernel<F32, OUT32, ANY, 128, 128><<<grid, 256, 0, s>>>(a, p.parts, part);
  }
}

template <bool F32, bool OUT32>
int linear_dispatch(const LinearArgs& a, const moe_linear_config& c, float* part, hipStream_t s) {
  // Offsets within a tile's rows are 32-bit byte offsets.
  if (std::max(a.ldx, a.ldw) >= (int64_t{1} << 23)) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.N, kAnyTile)), static_cast<unsigned>(ceil_div(a.M, kAnyTile)));
    linear_any_kernel<F32, OUT32><<<grid, 256, 0, s>>>(a);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
  }
  const int64_t unit = F32 ? 4 : 8;        // elements of 16 bytes
  const bool aligned = a.ldx % unit == 0 && a.ldw % unit == 0 && a.K % unit == 0 &&
                       reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.w) % 16 == 0;
  const LinearPlan p = linear_plan(c, a.M, !F32 && aligned && a.K % 128 == 0);
  if (p.rows == kWideRows) {
    if constexpr (!F32) {
      const unsigned grid = static_cast<unsigned>(std::min<int64_t>(kCus, ceil_div(p.tiles * p.parts, 8) * 8));
      if (p.cols == 256) linear_wide_kernel<OUT32, 256><<<grid, kWideThreads, 0, s>>>(a, p.parts, part);
      else linear_wide_kernel<OUT32, 128><<<grid, kWideThreads, 0, s>>>(a, p.parts, part);
    }
  } else if (aligned) {
    linear_launch<F32, OUT32, false>(a, p, part, s);
  } else {
    linear_launch<F32, OUT32, true>(a, p, part, s);
  }
  if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  if (p.parts > 1) {
    linear_finish_kernel<F32, OUT32><<<static_cast<unsigned>(ceil_div(a.M * part_stride(a.N) / 4, 256)), 256, 0, s>>>(
        a, p.parts, part);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_linear_workspace_size(const moe_linear_config* cfg, int32_t max_rows, size_t* bytes) {
  const int st = check_linear(cfg, max_rows);
  if (st) return st;
  if (!bytes) return MOE_ERR_NULL_PTR;
  *bytes = linear_workspace(*cfg, max_rows);
  return MOE_OK;
}

int moe_linear(const moe_linear_config* cfg, int32_t M, const void* x, int64_t ldx, const void* w, int64_t ldw,
               const void* bias, const void* residual, int64_t ldr, void* y, int64_t ldy, void* workspace,
               size_t workspace_bytes, void* stream) {
  const int st = check_linear(cfg, M);
  if (st) return st;
  if (M == 0) return MOE_OK;
  if (!x || !w || !y || !workspace) return MOE_ERR_NULL_PTR;
  const int64_t N = cfg->out_features, K = cfg->in_features;
  if (ldx < K || ldw < K || ldy < N || (residual && ldr < N)) return MOE_ERR_BAD_SHAPE;
  const int64_t far = int64_t{1} << 40;     // strides whose products with a row index stay in 64 bits
  if (ldx > far || ldw > far || ldy > far || (residual && ldr > far)) return MOE_ERR_UNSUPPORTED;
  if (residual == y && ldr != ldy) return MOE_ERR_BAD_SHAPE;
  if (workspace_bytes < linear_workspace(*cfg, M)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (off(x, cfg->in_dtype) || off(w, cfg->in_dtype) || off(bias, cfg->in_dtype) || off(residual, cfg->out_dtype) ||
      off(y, cfg->out_dtype) || reinterpret_cast<uintptr_t>(workspace) % 16)
    return MOE_ERR_UNSUPPORTED;
  LinearArgs a{};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.y = y;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldr = ldr;
  a.ldy = ldy;
  a.M = M;
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.act = cfg->activation;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  if (cfg->in_dtype == MOE_DTYPE_F32) return linear_dispatch<true, true>(a, *cfg, part, s);
  return cfg->out_dtype == MOE_DTYPE_F32 ? linear_dispatch<false, true>(a, *cfg, part, s)
                                         : linear_dispatch<false, false>(a, *cfg, part, s);
}

}  // extern "C"
