// Weight streaming for at most 16 activation rows (included by the kernels that use it).
//
// A wave multiplies 16 activation rows by a tile of 16 weight rows.  The weights go
// from global memory straight into the registers of the MFMA that uses them: every
// weight byte is used once, so a pass through LDS would move each byte twice for
// nothing.  Activations are the A operand (lane l: row l % 16), weights the B operand.
//
// A load instruction takes 128 bytes from each of 8 weight rows.  The plain operand
// layout (16 rows, 64 bytes each) reads at three quarters of that rate: 5.2 against
// 6.9 TB/s over 336 MB, 4.3 against 5.1 over 42 MB.  Lane l, with column c = l % 16 and
// lane group g = l / 16, loads row c % 8, 16-byte piece 4 (c / 8) + g.  To the MFMA the
// columns c < 8 are then the 8 rows over the first half of the 128 bytes and the
// columns c >= 8 the same rows over the second half, so each register meets the
// activations of both halves, in two accumulators of which half the columns count.
// That doubles the MFMAs, which are idle otherwise.
//
// A block is 128 bytes of each weight row: 64 bf16, 128 fp8 (one scale group), 256
// MXFP4 or 32 f32 elements.  The activations are taken in the order in which the lanes
// hold the weights, which is all that a sum needs.  Quantised weights are decoded to
// bf16, which holds every e4m3 and E2M1 value (and every E2M1 value times a power of
// two) exactly; the activations stay as they are.  The reason to quantise them
// elsewhere is the matrix cores' rate, and with 16 rows that rate is idle.
#pragma once

#include "kernels.h"
#include "schedule.h"

namespace moe {
namespace {

constexpr int kSkinnyRows = 16;

template <int FMT>
struct SkinnyFmt {
  static constexpr bool kF32 = FMT == kDtypeF32;
  static constexpr int kBlk = kF32 ? 32 : FMT == kDtypeBf16 ? 64 : FMT == kDtypeFp8 ? 128 : 256;   // elements
  static constexpr int kX = FMT == kDtypeMxfp4 ? 4 : FMT == kDtypeFp8 ? 2 : 1;   // activation pieces per half
};
constexpr int kBlkBytes = 128;   // of a weight row

// A lane's view of its two weight rows: rows c % 8 of the first and of the second 8
// of the tile, and their scales.
struct WRow {
  const uint8_t* p[2];
  const void* s[2];
};

// One block of a tile, as loaded.
template <int FMT>
struct WBlk {
  uint4 v[2];
  float s[2];     // fp8 group scale, or 2^(e - 127) of the lane's MXFP4 block
};
template <int FMT>
struct XBlk {
  uint4 v[2][SkinnyFmt<FMT>::kX];   // the two halves of the block
};
// Sums of a tile's two row sets over the two halves.
struct Acc {
  f32x4 v[2][2];
};

// Four floats at element k of a row of `kdim`, zeros past its end.
__device__ __forceinline__ uint4 ld_f32x4(const float* row, int k, int kdim, bool vec) {
  if (vec) return k < kdim ? ld16(row + k) : uint4{0, 0, 0, 0};
  uint4 r;
  r.x = k + 0 < kdim ? __float_as_uint(row[k + 0]) : 0;
  r.y = k + 1 < kdim ? __float_as_uint(row[k + 1]) : 0;
  r.z = k + 2 < kdim ? __float_as_uint(row[k + 2]) : 0;
  r.w = k + 3 < kdim ? __float_as_uint(row[k + 3]) : 0;
  return r;
}

// Block b of a tile's weight rows.  kdim and vec matter to f32 only: the other types
// come in whole blocks, 16-byte aligned.
template <int FMT>
__device__ __forceinline__ void load_w(WBlk<FMT>& w, const WRow& r, int b, int lane, int kdim, bool vec) {
  const int piece = ((lane >> 1) & 4) + (lane >> 4);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kDtypeF32) {
      w.v[h] = ld_f32x4(reinterpret_cast<const float*>(r.p[h]), 32 * b + 4 * piece, kdim, vec);
    } else {
      w.v[h] = ld16_stream(r.p[h] + static_cast<size_t>(b) * kBlkBytes + 16 * piece);
      if constexpr (FMT == kDtypeFp8) w.s[h] = static_cast<const float*>(r.s[h])[b];
      if constexpr (FMT == kDtypeMxfp4)
        w.s[h] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint8_t*>(r.s[h])[8 * b + piece]) << 23);
    }
  }
}

// The activations that meet block b; zeros for a row that is not `live`.
template <int FMT>
__device__ __forceinline__ void load_x(XBlk<FMT>& x, const void* row, int b, int lane, int kdim, bool vec, bool live) {
  using F = SkinnyFmt<FMT>;
  const int g = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < F::kX; ++q) x.v[h][q] = uint4{0, 0, 0, 0};
  if (!live) return;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < F::kX; ++q) {
      if constexpr (FMT == kDtypeF32)
        x.v[h][q] = ld_f32x4(static_cast<const float*>(row), 32 * b + 16 * h + 4 * g, kdim, vec);
      else
        x.v[h][q] = ld16(static_cast<const uint8_t*>(row) +
                         2 * (static_cast<size_t>(b) * F::kBlk + h * (F::kBlk / 2) + g * (F::kBlk / 8) + 8 * q));
    }
}

// The bf16 B operand that meets activation piece q, decoded from a loaded piece.
template <int FMT>
__device__ __forceinline__ uint4 decode_w(const uint4& v, float s, int q) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if constexpr (FMT == kDtypeBf16) {
    return v;
  } else if constexpr (FMT == kDtypeFp8) {
    const uint32_t lo = q ? v.z : v.x, hi = q ? v.w : v.y;
    const bf16x2 r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true)};
    return __builtin_bit_cast(uint4, r);
  } else {
    const uint32_t d = q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
    const bf16x2 r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3)};
    return __builtin_bit_cast(uint4, r);
  }
}

// acc += (the sum of N activation planes) * w over one block, without fp8 scales.
template <int FMT, int N>
__device__ __forceinline__ void mma_planes(const XBlk<FMT> (&x)[N], const WBlk<FMT>& w, Acc& acc) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kDtypeF32) {
      const float wv[4] = {__uint_as_float(w.v[h].x), __uint_as_float(w.v[h].y), __uint_as_float(w.v[h].z),
                           __uint_as_float(w.v[h].w)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 xv = x[0].v[k][0];
        const float xs[4] = {__uint_as_float(xv.x), __uint_as_float(xv.y), __uint_as_float(xv.z), __uint_as_float(xv.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc.v[h][k] = __builtin_amdgcn_mfma_f32_16x16x4f32(xs[i], wv[i], acc.v[h][k], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int q = 0; q < SkinnyFmt<FMT>::kX; ++q) {
        const uint4 wq = decode_w<FMT>(w.v[h], w.s[h], q);
#pragma unroll
        for (int p = N - 1; p >= 0; --p)      // the smallest plane first
#pragma unroll
          for (int k = 0; k < 2; ++k) acc.v[h][k] = mfma_bf16_16x16x32(x[p].v[k][q], wq, acc.v[h][k]);
      }
    }
  }
}

// acc += x * w over one block.
template <int FMT>
__device__ __forceinline__ void mma_block(const XBlk<FMT> (&x)[1], const WBlk<FMT>& w, Acc& acc) {
  if constexpr (FMT == kDtypeFp8) {
    Acc t{};
    mma_planes<FMT, 1>(x, w, t);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[h][k][i] = fmaf(t.v[h][k][i], w.s[h], acc.v[h][k][i]);
  } else {
    mma_planes<FMT, 1>(x, w, acc);
  }
}

// The tile's sums, the two halves added: element i of lane l is weight row l % 16 of
// the tile and activation row 4 (l / 16) + i.
__device__ __forceinline__ f32x4 tile_sums(const Acc& acc, int lane) {
  const bool upper = lane & 8;       // row set 1, and the columns that hold second halves
  f32x4 s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float give = upper ? acc.v[0][1][i] : acc.v[1][0][i];
    const float own = upper ? acc.v[1][1][i] : acc.v[0][0][i];
    s[i] = own + __shfl_xor(give, 8, kWave);
  }
  return s;
}

// Runs n blocks in batches of D: the loads of a batch are issued together, then its
// blocks are used.  A wave waits for a whole batch; its neighbours on the CU fill that
// time (a ring that keeps loads in flight across batches needed more registers, which
// halved the waves, and ran slower).  issue and use step their own position.
template <int D, class B, class Issue, class Use>
__device__ __forceinline__ void batches(int n, Issue issue, Use use) {
  for (int c = 0; c < n; c += D) {
    B b[D];
#pragma unroll
    for (int s = 0; s < D; ++s)
      if (c + s < n) issue(b[s]);
#pragma unroll
    for (int s = 0; s < D; ++s)
      if (c + s < n) use(b[s]);
  }
}

}  // namespace
}  // namespace moe
