// Matrices laid out afresh, for products that take whole 16-byte pieces.
#pragma once

#include "common.h"

namespace moe {
namespace {

// Matrices of one element size copied to rows of whole 16-byte pieces, zeros behind the
// columns and the rows: 16-bit elements, or bytes.
struct PackItem {
  const void* src;
  void* dst;
  int64_t ld, dst_ld;            // elements; dst_ld of whole pieces
  int rows, cols, dst_rows;
};
constexpr int kPackItems = 5;
struct PackArgs {
  PackItem item[kPackItems];
  int n;
};
// Row `row` of an item, by a workgroup.
template <class T>
__device__ __forceinline__ void pack_row(const PackItem& p, int64_t row) {
  constexpr int kPiece = 16 / sizeof(T);
  const T* src = static_cast<const T*>(p.src) + row * p.ld;
  const int cols = row < p.rows ? p.cols : 0;
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4), aligned(1)));
  for (int i = kPiece * threadIdx.x; i < p.dst_ld; i += kPiece * blockDim.x) {
    uint4 v = {0, 0, 0, 0};
    if (i + kPiece <= cols) {
      const u32x4_t q = *reinterpret_cast<const u32x4_t*>(src + i);
      v = uint4{q.x, q.y, q.z, q.w};
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < kPiece; ++e)
        if (i + e < cols) w[e * sizeof(T) / 4] |= static_cast<uint32_t>(src[i + e]) << (8 * sizeof(T) * (e % (4 / sizeof(T))));
      v = uint4{w[0], w[1], w[2], w[3]};
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(p.dst) + row * p.dst_ld + i) = v;
  }
}
template <class T>
__global__ void __launch_bounds__(256) pack_rows_kernel(PackArgs a) {
  int64_t row = blockIdx.x;
  int k = 0;
  while (k + 1 < a.n && row >= a.item[k].dst_rows) row -= a.item[k++].dst_rows;
  pack_row<T>(a.item[k], row);
}
template <class T>
inline bool pack_rows(const PackArgs& a, hipStream_t s) {
  int64_t rows = 0;
  for (int k = 0; k < a.n; ++k) rows += a.item[k].dst_rows;
  if (rows == 0) return true;
  pack_rows_kernel<T><<<static_cast<unsigned>(rows), 256, 0, s>>>(a);
  return hipGetLastError() == hipSuccess;
}

}  // namespace
}  // namespace moe
