// What the dense products share: activations, loads and stores of a few neighbouring
// elements at any alignment, and the order of the tiles on the chip's XCDs.
#pragma once

#include "moe_mi355x.h"
#include "skinny.h"

namespace moe {
namespace {

// Floats between rows of a plane of partial sums.
__host__ __device__ inline int64_t part_stride(int64_t N) { return (N + 3) / 4 * 4; }

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

// The first `left` of four neighbouring elements as they lie in memory, zeros behind them.
template <bool F32>
struct Raw4 {
  uint32_t v[F32 ? 4 : 2];
};
template <bool F32>
__device__ __forceinline__ Raw4<F32> raw4(const void* p, size_t i, int left) {
  typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
  typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(4)));
  Raw4<F32> r;
  if constexpr (F32) {
    const uint32_t* q = static_cast<const uint32_t*>(p) + i;
    if (left >= 4) {
      const u32x4_any v = *reinterpret_cast<const u32x4_any*>(q);
#pragma unroll
      for (int c = 0; c < 4; ++c) r.v[c] = v[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) r.v[c] = c < left ? q[c] : 0u;
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (left >= 4) {
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(q);
      r.v[0] = v.x;
      r.v[1] = v.y;
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        r.v[c] = (2 * c < left ? q[2 * c] : 0u) | (2 * c + 1 < left ? static_cast<uint32_t>(q[2 * c + 1]) << 16 : 0u);
    }
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ float value4(const Raw4<F32>& r, int c) {
  if constexpr (F32) return __uint_as_float(r.v[c]);
  else return __uint_as_float((c & 1) ? r.v[c >> 1] & 0xffff0000u : r.v[c >> 1] << 16);
}
// The first `left` of four elements.
template <bool F32>
__device__ __forceinline__ void put4(void* p, size_t i, const float* v, int left) {
  if (left >= 4) {
    store4<F32>(p, i, v);
    return;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c < left) {
      if constexpr (F32) static_cast<float*>(p)[i + c] = v[c];
      else static_cast<uint16_t*>(p)[i + c] = f32_to_bf16_bits(v[c]);
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

// Tile of workgroup b of 8 ceil(total / 8), or -1: tiles that share rows of W are
// neighbours on one XCD (workgroup b runs on XCD b % 8).
__device__ __forceinline__ int xcd_tile(int b, int total) {
  const int per = (total + 7) / 8;
  return b / 8 < per && (b % 8) * per + b / 8 < total ? (b % 8) * per + b / 8 : -1;
}

}  // namespace
}  // namespace moe
