// What the kernels that work on whole rows share: loads and stores of eight neighbouring
// elements at any alignment, sums and maxima over a row's lanes, and the 8-bit codes.
#pragma once

#include "common.h"

namespace moe {
namespace {

// Eight elements as they lie in memory (global accesses of 16 bytes need no alignment).
typedef uint32_t u32x4_row __attribute__((ext_vector_type(4), aligned(2)));
template <bool F32>
struct Raw8 {
  u32x4 v[F32 ? 2 : 1];
};

// The first `left` of the eight elements from p[i] on, zeros behind them.
template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* p, int i, int left) {
  Raw8<F32> r;
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + i;
    if (left >= 8) {
      r.v[0] = *reinterpret_cast<const u32x4_row*>(q);
      r.v[1] = *reinterpret_cast<const u32x4_row*>(q + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e >> 2][e & 3] = e < left ? __float_as_uint(q[e]) : 0u;
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (left >= 8) {
      r.v[0] = *reinterpret_cast<const u32x4_row*>(q);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r.v[0][e] = (2 * e < left ? q[2 * e] : 0u) | (2 * e + 1 < left ? static_cast<uint32_t>(q[2 * e + 1]) << 16 : 0u);
    }
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ float value(const Raw8<F32>& r, int e) {
  if constexpr (F32) return __uint_as_float(r.v[e >> 2][e & 3]);
  else return __uint_as_float((e & 1) ? r.v[0][e >> 1] & 0xffff0000u : r.v[0][e >> 1] << 16);
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8], int left) {
  Raw8<F32> r;
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e >> 2][e & 3] = __float_as_uint(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[0][e] = f32_to_bf16_bits(v[2 * e]) | static_cast<uint32_t>(f32_to_bf16_bits(v[2 * e + 1])) << 16;
  }
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + i;
    if (left >= 8) {
      *reinterpret_cast<u32x4_row*>(q) = r.v[0];
      *reinterpret_cast<u32x4_row*>(q + 4) = r.v[1];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) q[e] = v[e];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if (left >= 8) {
      *reinterpret_cast<u32x4_row*>(q) = r.v[0];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) q[e] = static_cast<uint16_t>(r.v[0][e >> 1] >> (16 * (e & 1)));
    }
  }
}
// Eight elements whose type only the launch knows.
__device__ __forceinline__ void load8_of(bool f32, const void* p, int i, int left, float (&v)[8]) {
  if (f32) {
    const Raw8<true> r = load8<true>(p, i, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = value<true>(r, e);
  } else {
    const Raw8<false> r = load8<false>(p, i, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = value<false>(r, e);
  }
}
__device__ __forceinline__ float load_of(bool f32, const void* p, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store_of(bool f32, void* p, int64_t i, float v) {
  if (f32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = f32_to_bf16_bits(v);
}

// ---------------------------------------------------------------- over the wave

// Rotations within 16 lanes, then the two halves of 32 and of 64 swapped: every lane
// combines equal operands in every step, so all get the same bits.
template <class T, class F>
__device__ __forceinline__ T sixteen_all(T x, F f) {
  const auto step = [&](auto rotated) { x = f(x, __builtin_bit_cast(T, rotated)); };
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xf, 0xf, true));   // row_ror:8
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x124, 0xf, 0xf, true));
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x122, 0xf, 0xf, true));
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x121, 0xf, 0xf, true));
  return x;
}
template <class T, class F>
__device__ __forceinline__ T wave_all(T x, F f) {
  x = sixteen_all(x, f);
  const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x), false, false);
  x = f(__builtin_bit_cast(T, static_cast<unsigned>(a[0])), __builtin_bit_cast(T, static_cast<unsigned>(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, x), false, false);
  return f(__builtin_bit_cast(T, static_cast<unsigned>(b[0])), __builtin_bit_cast(T, static_cast<unsigned>(b[1])));
}

// N sums (or maxima) over the `waves` waves of a row, in every lane.  The waves meet in
// one of two buffers by turns: a wave that writes a buffer again has passed the barrier
// of the other one in between, behind which nobody reads the first.
constexpr int kRowWaves = 16, kRowValues = 4;
template <class T>
struct RowLds {
  T v[2][kRowValues][kRowWaves];
};
template <int N, class T, class F>
__device__ __forceinline__ void row_all(T (&v)[N], int wave, int waves, RowLds<T>& lds, int& turn, F f) {
  static_assert(N <= kRowValues, "buffer");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_all(v[i], f);
  if (waves == 1) return;
#pragma unroll
  for (int i = 0; i < N; ++i) lds.v[turn][i][wave] = v[i];     // every lane the same value
  __syncthreads();
  // Lane l takes wave l % 16's value (a sum's or a magnitude's identity is 0).
  const int w = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = w < waves ? lds.v[turn][i][w] : T(0);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = sixteen_all(v[i], f);
  turn ^= 1;
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Most {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// ---------------------------------------------------------------- 8-bit codes

// A row's scale from the bits of its largest magnitude, max(amax / 127, 2^-126); a row
// with an infinity or a NaN has that as its scale, and codes of 0.
__device__ __forceinline__ float i8_scale(uint32_t amax) {
  return amax >= 0x7f800000u ? __uint_as_float(amax) : fmaxf(__uint_as_float(amax) / 127.0f, 0x1p-126f);
}
// x / s rounded to the nearest whole number, ties to even, where x (1 / s) may land on the
// wrong side of a border; x - (q -+ 1/2) s, rounded once, has its sign right.
__device__ __forceinline__ float i8_border(float x, float s, float q) {
  const float lo = fmaf(0.5f - q, s, x), hi = fmaf(-0.5f - q, s, x);
  const bool odd = static_cast<int>(q) & 1;
  return lo < 0.0f || (lo == 0.0f && odd) ? q - 1.0f : hi > 0.0f || (hi == 0.0f && odd) ? q + 1.0f : q;
}
// Codes of eight elements.  |x / s| <= 127 (1 + 2^-24), so x (1 / s) is off by less than
// 2^-15: only quotients within that of a border, a few in a hundred thousand, are decided
// by the exact remainder.
__device__ __forceinline__ void store_codes(int8_t* p, const float (&v)[8], float s, float inv, int left) {
  uint32_t w[2] = {0, 0};
  if (inv > 0.0f) {                            // else a scale of inf or NaN
    float q[8], far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = v[e] * inv;
      q[e] = rintf(t);
      far = fmaxf(far, fabsf(t - q[e]));
    }
    if (far > 0.5f - 0x1p-14f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = i8_border(v[e], s, q[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e >> 2] |= (static_cast<uint32_t>(static_cast<int>(q[e])) & 0xffu) << (8 * (e & 3));
  }
  if (left >= 8) {
    typedef uint32_t u32x2_b __attribute__((ext_vector_type(2), aligned(1)));
    *reinterpret_cast<u32x2_b*>(p) = u32x2_b{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3)));
  }
}

}  // namespace
}  // namespace moe
