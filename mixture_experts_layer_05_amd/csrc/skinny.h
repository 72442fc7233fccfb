// Weight streaming for at most 16 activation rows (included by the kernels that use it).
//
// A wave multiplies 16 activation rows by tiles of 16 weight rows.  The weight
// fragments go from global memory straight into the registers of the MFMA that
// uses them: every weight byte is used once, so a pass through LDS would move each
// byte twice for nothing.  Activations are the A operand (lane l: row l % 16),
// weights the B operand (lane l: weight row l % 16), so a lane's accumulators all
// belong to one weight row and a weight row's scale is one register.
//
// The contraction runs in blocks.  In a block lane group g = l / 16 takes 16-byte
// pieces of its weight row; the activations are taken in the same order, which is
// all that the sum needs:
//   bf16   128 elements: piece q (4) holds elements 32 q + 8 g .. + 8
//   fp8    128 elements (one scale group): piece q (2) holds 64 q + 16 g .. + 16
//   MXFP4  128 elements: the piece holds 32 g .. + 32, one E8M0 block
//   f32    32 elements: piece q (2) holds 16 q + 4 g .. + 4
// Quantised weights are decoded to bf16, which holds every e4m3 and E2M1 value (and
// every E2M1 value times a power of two) exactly; the activations stay as they are.
// The reason to quantise them elsewhere is the matrix cores' rate, and with 16 rows
// that rate is idle.
#pragma once

#include "kernels.h"
#include "schedule.h"

namespace moe {
namespace {

constexpr int kSkinnyRows = 16;

template <int FMT>
struct SkinnyFmt {
  static constexpr bool kF32 = FMT == kDtypeF32;
  static constexpr int kBlk = kF32 ? 32 : 128;                                  // elements per block
  static constexpr int kW = FMT == kDtypeBf16 ? 4 : FMT == kDtypeMxfp4 ? 1 : 2;  // weight pieces per lane
  static constexpr int kX = kF32 ? 2 : 4;                                       // activation pieces per lane
  static constexpr int kWBytes = kF32 ? 128 : FMT == kDtypeBf16 ? 256 : FMT == kDtypeFp8 ? 128 : 64;
  static constexpr int kXBytes = kF32 ? 128 : 256;
};

// A lane's view of one weight row: its first byte and its scales.
struct WRow {
  const uint8_t* p;
  const void* s;
};

// One block of one 16-row weight tile, as loaded.
template <int FMT>
struct WBlk {
  uint4 v[SkinnyFmt<FMT>::kW];
  float s;        // fp8 group scale, or 2^(e - 127) of the lane's MXFP4 block
};
template <int FMT>
struct XBlk {
  uint4 v[SkinnyFmt<FMT>::kX];
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

// Block b of a weight row (g: the lane group).  kdim and vec matter to f32 only: the
// other types come in whole blocks, 16-byte aligned.
template <int FMT>
__device__ __forceinline__ void load_w(WBlk<FMT>& w, const WRow& r, int b, int g, int kdim, bool vec) {
  using F = SkinnyFmt<FMT>;
  if constexpr (FMT == kDtypeF32) {
#pragma unroll
    for (int q = 0; q < F::kW; ++q)
      w.v[q] = ld_f32x4(reinterpret_cast<const float*>(r.p), 32 * b + 16 * q + 4 * g, kdim, vec);
  } else {
    const uint8_t* p = r.p + static_cast<size_t>(b) * F::kWBytes + 16 * g;
#pragma unroll
    for (int q = 0; q < F::kW; ++q) w.v[q] = ld16_stream(p + 64 * q);
    if constexpr (FMT == kDtypeFp8) w.s = static_cast<const float*>(r.s)[b];
    if constexpr (FMT == kDtypeMxfp4)
      w.s = __uint_as_float(static_cast<uint32_t>(static_cast<const uint8_t*>(r.s)[4 * b + g]) << 23);
  }
}

// The activations that meet block b; zeros for a row that is not `live`.
template <int FMT>
__device__ __forceinline__ void load_x(XBlk<FMT>& x, const void* row, int b, int g, int kdim, bool vec, bool live) {
  using F = SkinnyFmt<FMT>;
#pragma unroll
  for (int q = 0; q < F::kX; ++q) x.v[q] = uint4{0, 0, 0, 0};
  if (!live) return;
  if constexpr (FMT == kDtypeF32) {
#pragma unroll
    for (int q = 0; q < F::kX; ++q)
      x.v[q] = ld_f32x4(static_cast<const float*>(row), 32 * b + 16 * q + 4 * g, kdim, vec);
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(row) + static_cast<size_t>(b) * F::kXBytes;
#pragma unroll
    for (int q = 0; q < F::kX; ++q) {
      const int at = FMT == kDtypeBf16 ? 64 * q + 16 * g
                   : FMT == kDtypeFp8 ? 128 * (q >> 1) + 32 * g + 16 * (q & 1)
                                      : 64 * g + 16 * q;
      x.v[q] = ld16(p + at);
    }
  }
}

// bf16 B operand of the block's q-th MFMA (q < 4), decoded from the loaded pieces.
template <int FMT>
__device__ __forceinline__ uint4 decode_w(const WBlk<FMT>& w, int q) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if constexpr (FMT == kDtypeBf16) {
    return w.v[q];
  } else if constexpr (FMT == kDtypeFp8) {
    const uint4 v = w.v[q >> 1];
    const uint32_t lo = (q & 1) ? v.z : v.x, hi = (q & 1) ? v.w : v.y;
    const bf16x2 r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true)};
    return __builtin_bit_cast(uint4, r);
  } else {
    const uint32_t d = q == 0 ? w.v[0].x : q == 1 ? w.v[0].y : q == 2 ? w.v[0].z : w.v[0].w;
    const bf16x2 r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, w.s, 0),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, w.s, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, w.s, 2),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, w.s, 3)};
    return __builtin_bit_cast(uint4, r);
  }
}

// acc += x * w over one block, before any fp8 scale.
template <int FMT>
__device__ __forceinline__ f32x4 mma_raw(const XBlk<FMT>& x, const WBlk<FMT>& w, f32x4 acc) {
  if constexpr (FMT == kDtypeF32) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.v[q].x), __uint_as_float(w.v[q].x), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.v[q].y), __uint_as_float(w.v[q].y), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.v[q].z), __uint_as_float(w.v[q].z), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.v[q].w), __uint_as_float(w.v[q].w), acc, 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc = mfma_bf16_16x16x32(x.v[q], decode_w<FMT>(w, q), acc);
  }
  return acc;
}

// acc += x * w over one block.
template <int FMT>
__device__ __forceinline__ void mma_block(const XBlk<FMT>& x, const WBlk<FMT>& w, f32x4& acc) {
  if constexpr (FMT == kDtypeFp8) {
    const f32x4 t = mma_raw<FMT>(x, w, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(t[i], w.s, acc[i]);
  } else {
    acc = mma_raw<FMT>(x, w, acc);
  }
}

// Runs n blocks through two register buffers, a block's loads issued two blocks
// before its use.  In the main loop every issue is unconditional: where two paths
// with and without a load meet, the compiler can only wait for everything.
template <class B, class Issue, class Use>
__device__ __forceinline__ void two_ahead(int n, Issue issue, Use use) {
  if (n <= 0) return;
  B b0, b1;
  issue(0, b0);
  if (n == 1) {
    use(0, b0);
    return;
  }
  issue(1, b1);
  int i = 0;
  for (; i + 3 < n; i += 2) {
    use(i, b0);
    issue(i + 2, b0);
    use(i + 1, b1);
    issue(i + 3, b1);
  }
  use(i, b0);
  if (i + 2 < n) {          // three left
    issue(i + 2, b0);
    use(i + 1, b1);
    use(i + 2, b0);
  } else {
    use(i + 1, b1);
  }
}

}  // namespace
}  // namespace moe
