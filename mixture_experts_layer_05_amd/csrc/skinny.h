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
// lane group g = l / 16, loads row c % 8, 16-byte piece 4 (c / 8) + g, of the first 8
// rows and of the second 8.  Lanes c and c ^ 8 then exchange one register each, which
// gives both the operands of row c: its first and its second 64 bytes.
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

// The matrices of a tile's first and second 8 rows, and their scales.
struct Matrices {
  const void *w[2], *s[2];
};
// A lane's view of a tile: offsets of its piece of block 0 in rows c % 8 of the first
// and of the second 8, and the scales of the tile's row c (the row whose operands the
// lane holds after the trade).
struct WRow {
  uint32_t w[2];
  const uint8_t* s;
};

// One block of a tile, as loaded.
template <int FMT>
struct WBlk {
  uint4 v[2];
  uint2 s;        // fp8: the row's group scale; MXFP4: its 8 E8M0 codes
};
template <int FMT>
struct XBlk {
  uint4 v[2][SkinnyFmt<FMT>::kX];   // the two halves of the block
};

template <int FMT>
__host__ __device__ constexpr size_t row_bytes(int k) {
  return FMT == kDtypeF32 ? static_cast<size_t>(k) * 4
       : FMT == kDtypeBf16 ? static_cast<size_t>(k) * 2
       : FMT == kDtypeFp8 ? static_cast<size_t>(k) : static_cast<size_t>(k) / 2;
}
template <int FMT>
__host__ __device__ constexpr size_t scale_bytes(int k) {
  return FMT == kDtypeFp8 ? static_cast<size_t>(k) / kGroup * 4
       : FMT == kDtypeMxfp4 ? static_cast<size_t>(k) / kMxBlock : 0;
}

// A lane's 16-byte piece of its block.
__device__ __forceinline__ int lane_piece(int lane) { return ((lane >> 1) & 4) + (lane >> 4); }

// Rows row0 and row1, of k elements, of the first and the second matrix are the lane's
// rows c % 8.  A matrix is smaller than 4 GiB.
template <int FMT>
__device__ __forceinline__ WRow weight_rows(const Matrices& m, int row0, int row1, int k, int lane) {
  WRow r;
  const uint32_t bytes = static_cast<uint32_t>(row_bytes<FMT>(k));
  r.w[0] = static_cast<uint32_t>(row0) * bytes + 16 * lane_piece(lane);
  r.w[1] = static_cast<uint32_t>(row1) * bytes + 16 * lane_piece(lane);
  r.s = static_cast<const uint8_t*>((lane & 8) ? m.s[1] : m.s[0]) +
        static_cast<size_t>((lane & 8) ? row1 : row0) * scale_bytes<FMT>(k);
  return r;
}

// Four floats, of which the row holds the first n (vec: 16-byte aligned, all or none).
__device__ __forceinline__ uint4 ld_f32x4(const uint8_t* p, int n, bool vec) {
  uint4 r = {0, 0, 0, 0};
  if (vec) {
    if (n > 0) r = ld16(p);
    return r;
  }
  const uint32_t* f = reinterpret_cast<const uint32_t*>(p);
  if (n > 0) r.x = f[0];
  if (n > 1) r.y = f[1];
  if (n > 2) r.z = f[2];
  if (n > 3) r.w = f[3];
  return r;
}

// The scales of a lane's row for the D blocks from the one at `p` on, of which the row
// holds `left`.  They come several blocks to a load: a load of one block's scale takes
// a whole line from the L2 for each of the 16 rows, half as much again as the weights
// (256 experts, top-8, I 2048, H 7168, 16 tokens, fp8: 664 us with such loads,
// 568 with four blocks to a load, 541 without the scales).
template <int FMT, int D>
struct Scales {
  static constexpr bool kAny = FMT == kDtypeFp8 || FMT == kDtypeMxfp4;
  static constexpr int kInts = FMT == kDtypeMxfp4 ? 2 : 1;          // of a block
  static constexpr int kN = kAny ? D * kInts : 1;
  uint32_t v[kN];
  __device__ __forceinline__ void load(const uint8_t* p, int left) {
    if constexpr (kAny) {
      typedef uint32_t u32_any __attribute__((aligned(1)));
      typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
      typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
      if (left >= D) {
        constexpr int kQuads = kN / 4, kRest = kN % 4;
        static_assert(kRest != 3, "pieces of 4, 2 and 1");
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          const u32x4_any t = *reinterpret_cast<const u32x4_any*>(p + 16 * q);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * q + i] = t[i];
        }
        if constexpr (kRest == 2) {
          const u32x2_any t = *reinterpret_cast<const u32x2_any*>(p + 16 * kQuads);
          v[kN - 2] = t[0];
          v[kN - 1] = t[1];
        }
        if constexpr (kRest == 1) v[kN - 1] = *reinterpret_cast<const u32_any*>(p + 16 * kQuads);
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = i < left * kInts ? *reinterpret_cast<const u32_any*>(p + 4 * i) : 0;
      }
    }
  }
  __device__ __forceinline__ uint2 block(int d) const {
    if constexpr (!kAny) return uint2{0, 0};
    else return uint2{v[d * kInts], kInts == 2 ? v[d * kInts + kInts - 1] : 0};
  }
  // The next block's become the first.
  __device__ __forceinline__ void step() {
#pragma unroll
    for (int i = 0; i + kInts < kN; ++i) v[i] = v[i + kInts];
  }
};
// Bytes of a block's scales in a row.
template <int FMT>
__device__ __forceinline__ constexpr int blk_scale_bytes() {
  return FMT == kDtypeFp8 ? 4 : FMT == kDtypeMxfp4 ? 8 : 0;
}

// Block b of a tile's weight rows, without its scales.  kdim and vec matter to f32 only: the other types
// come in whole blocks, 16-byte aligned.
template <int FMT>
__device__ __forceinline__ void load_w(WBlk<FMT>& k, const Matrices& m, const WRow& r, int b, int lane, int kdim,
                                       bool vec) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t* wb = static_cast<const uint8_t*>(m.w[h]) + static_cast<size_t>(b) * kBlkBytes;
    if constexpr (FMT == kDtypeF32) k.v[h] = ld_f32x4(wb + r.w[h], kdim - 32 * b - 4 * lane_piece(lane), vec);
    else k.v[h] = ld16_stream(wb + r.w[h]);
  }
}

// The activations that meet block b, of the row at byte `off` from x; zeros for a row
// that is not `live`.
template <int FMT>
__device__ __forceinline__ void load_x(XBlk<FMT>& k, const void* x, uint32_t off, int b, int lane, int kdim, bool vec,
                                       bool live) {
  using F = SkinnyFmt<FMT>;
  const int g = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < F::kX; ++q) k.v[h][q] = uint4{0, 0, 0, 0};
  if (!live) return;
  const uint8_t* xb = static_cast<const uint8_t*>(x) + static_cast<size_t>(b) * F::kBlk * (F::kF32 ? 4 : 2);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < F::kX; ++q) {
      if constexpr (FMT == kDtypeF32)
        k.v[h][q] = ld_f32x4(xb + off + 4 * (16 * h + 4 * g), kdim - 32 * b - 16 * h - 4 * g, vec);
      else
        k.v[h][q] = ld16(xb + off + 2 * (h * (F::kBlk / 2) + g * (F::kBlk / 8) + 8 * q));
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

// (a, b) of lanes c < 8 and (a', b') of lanes c + 8 become (a, a') and (b, b').
__device__ __forceinline__ void trade(uint32_t& a, uint32_t& b, bool upper) {
  const uint32_t give = upper ? a : b;
  const uint32_t got = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(give), 0x128, 0xf, 0xf, true));   // row_ror:8, lane ^ 8
  a = upper ? got : a;
  b = upper ? b : got;
}

// acc += (the sum of N activation planes) * w over one block; element i of lane l is
// weight row l % 16 of the tile and activation row 4 (l / 16) + i.
template <int FMT, int N>
__device__ __forceinline__ f32x4 mma_planes(const XBlk<FMT> (&x)[N], WBlk<FMT> w, int lane, f32x4 acc) {
  const bool upper = lane & 8;
  trade(w.v[0].x, w.v[1].x, upper);
  trade(w.v[0].y, w.v[1].y, upper);
  trade(w.v[0].z, w.v[1].z, upper);
  trade(w.v[0].w, w.v[1].w, upper);
  if constexpr (FMT == kDtypeF32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 xv = x[0].v[h][0], wv = w.v[h];
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(xv.x), __uint_as_float(wv.x), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(xv.y), __uint_as_float(wv.y), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(xv.z), __uint_as_float(wv.z), acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(xv.w), __uint_as_float(wv.w), acc, 0, 0, 0);
    }
    return acc;
  } else {
    // 2^(e - 127) of the lane's E8M0 blocks, code g of either half: the conversion takes a
    // scale's exponent field, so 0.0f stands for 2^-127 and inf (code 255) gives NaN.
    float e8[2] = {0.f, 0.f};
    if constexpr (FMT == kDtypeMxfp4) {
      const int at = 8 * (lane >> 4);
      e8[0] = __uint_as_float(((w.s.x >> at) & 0xffu) << 23);
      e8[1] = __uint_as_float(((w.s.y >> at) & 0xffu) << 23);
    }
    f32x4 t = FMT == kDtypeFp8 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < SkinnyFmt<FMT>::kX; ++q) {
        const uint4 wq = decode_w<FMT>(w.v[h], e8[h], q);
#pragma unroll
        for (int p = N - 1; p >= 0; --p) t = mfma_bf16_16x16x32(x[p].v[h][q], wq, t);   // the smallest plane first
      }
    if constexpr (FMT == kDtypeFp8) {
      const float s = __uint_as_float(w.s.x);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = fmaf(t[i], s, acc[i]);
    }
    return t;
  }
}

// Runs n blocks in batches of D: the loads of a batch are issued together, then its
// blocks are used.  A wave waits for a whole batch; its neighbours on the CU fill that
// time.  issue and use step their own position; first() runs once, when the first
// batch's loads have been issued.
template <int D, class B, class Issue, class Use, class First>
__device__ __forceinline__ void batches(int n, Issue issue, Use use, First first) {
  for (int c = 0; c < n; c += D) {
    B b[D];
#pragma unroll
    for (int s = 0; s < D; ++s)
      if (c + s < n) issue(b[s]);
    if (c == 0) first();
#pragma unroll
    for (int s = 0; s < D; ++s)
      if (c + s < n) use(b[s]);
  }
  if (n <= 0) first();
}

}  // namespace
}  // namespace moe
