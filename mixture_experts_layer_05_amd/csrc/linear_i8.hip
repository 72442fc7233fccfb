// Products in 8-bit integers with a scale for each row of either operand:
//   y = act(sx sw sum_k q[m, k] w[n, k] + bias) + residual
// The sum is exact in int32, however it is split; everything behind it is float32, rounded
// once to y's type.  Rows of x in 16 or 32 bits are quantised first (quant_i8_kernel), each by
// its largest magnitude.  8192 x 4096 x 7168 from bf16 takes 249 to 278 us, of which 32 to 38
// are the quantiser's; one row against 17408 x 5120 24 us, 21 from codes.
#include "gemm.h"
#include "pack.h"
#include "rows.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- quantiser

// A row of x to a workgroup: its largest magnitude, then its codes.  A lane keeps C times
// eight elements; what is left of a longer row is read again, from the caches.  Zeros
// behind the row up to `width` codes.  Bound by memory: 8192 x 7168 bf16 takes 32 to 38 us,
// 5.3 TB/s read and written at 33 (67 us with every code decided by the exact remainder).  Workgroups from
// M on lay out rows of the product's weights, if those lie odd: a launch less.
template <bool F32, int C>
__global__ void __launch_bounds__(1024) quant_i8_kernel(const void* x, int64_t ldx, int K, int8_t* q, int64_t ldq, int width, float* scale, int M, PackItem pack) {
  __shared__ RowLds<uint32_t> lds;
  const int64_t m = blockIdx.x;
  if (m >= M) return pack_row<uint8_t>(pack, m - M);
  const uint8_t* row = static_cast<const uint8_t*>(x) + m * ldx * (F32 ? 4 : 2);
  const int waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), step = 8 * blockDim.x;
  const int first = 8 * threadIdx.x;
  uint32_t most[1] = {0};
  const auto add = [&](const Raw8<F32>& r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) most[0] = max(most[0], __float_as_uint(value<F32>(r, e)) & 0x7fffffffu);
  };
  Raw8<F32> head[C];
#pragma unroll
  for (int c = 0; c < C; ++c) head[c] = load8<F32>(row, first + c * step, K - first - c * step);
#pragma unroll
  for (int c = 0; c < C; ++c) add(head[c]);
  for (int i = first + C * step; i < K; i += step) add(load8<F32>(row, i, K - i));
  int turn = 0;
  row_all(most, wave, waves, lds, turn, Most{});
  const float s = i8_scale(most[0]), inv = 1.0f / s;
  if (threadIdx.x == 0) scale[m] = s;
  const auto put = [&](const Raw8<F32>& r, int i) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = value<F32>(r, e);
    if (i < width) store_codes(q + m * ldq + i, v, s, inv, width - i);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) put(head[c], first + c * step);
  for (int i = first + C * step; i < width; i += step) put(load8<F32>(row, i, K - i), i);
}

// Few elements: a lane for every eight, for the latency.  Many: four times as many to a
// lane, for the loads in flight and the workgroups on a CU.  Microseconds of the first and
// the second: 16 x 5120 3.0 and 4.8, 512 x 7168 4.8 and 5.7, 4096 x 1024 5.1 and 5.8,
// 1024 x 5120 6.2 and 6.5, 1024 x 7168 8.1 and 7.3, 4096 x 7168 24 and 18.
constexpr int64_t kFewElements = int64_t{6} << 20;
int quantise(bool f32, int M, int K, const void* x, int64_t ldx, int8_t* q, int64_t ldq, int width, float* scale, const PackItem& pack, hipStream_t s) {
  const bool few = static_cast<int64_t>(M) * K <= kFewElements;
  const unsigned block = 64u * static_cast<unsigned>(std::min<int64_t>(16, ceil_div(width, few ? 512 : 2048)));
  const unsigned grid = static_cast<unsigned>(M + pack.dst_rows);
  const auto launch = [&](auto kernel) { kernel<<<grid, block, 0, s>>>(x, ldx, K, q, ldq, width, scale, M, pack); };
  if (f32) few ? launch(quant_i8_kernel<true, 1>) : launch(quant_i8_kernel<true, 4>);
  else few ? launch(quant_i8_kernel<false, 1>) : launch(quant_i8_kernel<false, 4>);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
}

// ---------------------------------------------------------------- epilogue

template <bool OUT32>
struct I8Out {
  static constexpr int kAhead = OUT32 ? 4 : 8;
  struct Cols {
    float w[4], b[4];
  };
  struct Ahead {
    float sx;
    Raw4<OUT32> r;
  };
  const float *sx, *sw;
  const void *bias, *residual;
  void* y;
  int64_t ldr, ldy;
  int N, act;
  bool bias_f32;
  int bytes() const { return (OUT32 ? 4 : 2) * (residual ? 2 : 1); }
  __device__ __forceinline__ Cols cols(int n) const {
    Cols c;
    const Raw4<true> w = raw4<true>(sw, n, N - n);
    Raw4<true> b{};
    Raw4<false> h{};
    if (bias && bias_f32) b = raw4<true>(bias, n, N - n);
    if (bias && !bias_f32) h = raw4<false>(bias, n, N - n);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c.w[k] = value4<true>(w, k);
      c.b[k] = bias_f32 ? value4<true>(b, k) : value4<false>(h, k);
    }
    return c;
  }
  __device__ __forceinline__ Ahead ahead(int m, int n) const { return ahead(m, n, sx[m]); }
  __device__ __forceinline__ Ahead ahead(int m, int n, float scale) const {
    Ahead a{scale, {}};
    if (residual) a.r = raw4<OUT32>(residual, static_cast<size_t>(m) * ldr + n, N - n);
    return a;
  }
  __device__ __forceinline__ void put(int m, int n, const f32x4& s, const f32x4&, const Cols& c, const Ahead& a) const {
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = s[k] * a.sx * c.w[k] + c.b[k];
    activate<!OUT32>(v, act);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] += value4<OUT32>(a.r, k);
    put4<OUT32>(y, static_cast<size_t>(m) * ldy + n, v, N - n);
  }
};

// ---------------------------------------------------------------- one row, quantised on the way
//
// Every workgroup quantises the row for itself while its first weights are in flight; one
// of them also writes the scale, for the sums of parts.  It saves a launch, 1.5 to 2 us of
// 11 at 1 x 5120 x 5120, as long as the workgroups run in a round or two: with 17408
// columns it takes 30 us and two launches 27.  More rows, one after the other, take longer
// than a launch (4 x 5120 x 5120: 19 and 14).
template <bool F32>
struct QuantisedRow {
  static constexpr bool kStaged = true, kRests = false;
  const void* x;
  float* scale;
  int ld;                        // bytes of the codes in LDS, whole blocks; the scale behind them
  __device__ __forceinline__ void put(uint8_t* staged, int K, bool write) const {
    __shared__ RowLds<uint32_t> lds;
    const int tid = threadIdx.x, step = 8 * blockDim.x;
    Raw8<F32> head[2];
    uint32_t most[1] = {0};
    const auto add = [&](const Raw8<F32>& r) {
#pragma unroll
      for (int e = 0; e < 8; ++e) most[0] = max(most[0], __float_as_uint(value<F32>(r, e)) & 0x7fffffffu);
    };
#pragma unroll
    for (int c = 0; c < 2; ++c) head[c] = load8<F32>(x, 8 * tid + c * step, K - 8 * tid - c * step);
#pragma unroll
    for (int c = 0; c < 2; ++c) add(head[c]);
    for (int i = 8 * tid + 2 * step; i < K; i += step) add(load8<F32>(x, i, K - i));
    int turn = 0;
    row_all(most, tid >> 6, blockDim.x >> 6, lds, turn, Most{});
    const float s = i8_scale(most[0]), inv = 1.0f / s;
    if (tid == 0) {
      *reinterpret_cast<float*>(staged + ld) = s;
      if (write) *scale = s;
    }
    const auto codes = [&](const Raw8<F32>& r, int i) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = value<F32>(r, e);
      if (i < ld) store_codes(reinterpret_cast<int8_t*>(staged) + i, v, s, inv, 8);
    };
#pragma unroll
    for (int c = 0; c < 2; ++c) codes(head[c], 8 * tid + c * step);
    for (int i = 8 * tid + 2 * step; i < ld; i += step) codes(load8<F32>(x, i, K - i), i);
    __syncthreads();
  }
  template <class Epi>
  __device__ __forceinline__ typename Epi::Ahead ahead(const uint8_t* staged, const Epi& epi, int n) const {
    return epi.ahead(0, n, *reinterpret_cast<const float*>(staged + ld));
  }
};
constexpr int kOnTheWayBytes = 32 << 10, kOnTheWayColumns = 8192;

// ---------------------------------------------------------------- host

bool plain(int d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16; }
size_t size_of(int d) { return d == MOE_DTYPE_F32 ? 4 : d == MOE_DTYPE_BF16 ? 2 : 1; }
bool off(const void* p, size_t unit) { return reinterpret_cast<uintptr_t>(p) % unit != 0; }
constexpr int64_t kFar = int64_t{1} << 40;     // strides whose products with a row index stay in 64 bits

int check_i8(const moe_linear_i8_config* c, int32_t rows) {
  if (!c) return MOE_ERR_NULL_PTR;
  if ((!plain(c->in_dtype) && c->in_dtype != MOE_DTYPE_I8) || !plain(c->bias_dtype) || !plain(c->out_dtype)) return MOE_ERR_BAD_DTYPE;
  if (c->in_features <= 0 || c->out_features <= 0 || rows < 0) return MOE_ERR_BAD_SHAPE;
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_SILU) return MOE_ERR_BAD_SHAPE;
  if (c->in_features > MOE_I8_MAX_FEATURES || c->out_features > MOE_LINEAR_MAX_FEATURES || rows > MOE_LINEAR_MAX_ROWS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Codes that do not lie in whole 16-byte pieces are laid out afresh, in one launch, where
// the product is large: 300 x 2049 x 1025 takes 16.0 us with the codes as they lie and 14.5 so,
// 256 x 1023 x 515 18.5 and 11.7, 64 x 515 x 257 12.4 and 10.4, 64 x 257 x 257 10.7 and 11.1.
// Weights of whole pieces whose rows alone lie odd are taken as they lie, through registers
// (the workspace has no room for them): 1 x 4096 x 7168 from bf16 takes 16 us instead of 11,
// 224 x 4096 x 7168 31 instead of 22, 8192 x 4096 x 7168 384 to 402 instead of 249 to 262.
constexpr int64_t kPackFrom = int64_t{1} << 23;      // multiply-adds
bool large(const moe_linear_i8_config& c, int64_t M) { return M > kSkinnyRows && M * c.in_features * c.out_features >= kPackFrom; }

// The workspace: partial sums, then the codes of x in rows of whole 128-byte lines, their
// scales, and where rows of that length do not end with a 16-byte piece, room for w's codes.
int64_t codes_ld(const moe_linear_i8_config& c) { return align_up(c.in_features, 128); }
size_t codes_bytes(const moe_linear_i8_config& c, int64_t rows) { return align_up(static_cast<size_t>(rows) * codes_ld(c), 256); }
size_t i8_workspace(const moe_linear_i8_config& c, int64_t M) {
  return part_bytes(false, M, c.out_features) + codes_bytes(c, M) + align_up(M * 4, 256) +
         (c.in_features % 16 ? codes_bytes(c, c.out_features) : 0);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_quant_i8(int32_t dtype, int32_t rows, int32_t columns, const void* x, int64_t ldx, int8_t* codes, int64_t ldc,
                 float* scale, void* stream) {
  if (!plain(dtype)) return MOE_ERR_BAD_DTYPE;
  if (rows < 0 || columns <= 0) return MOE_ERR_BAD_SHAPE;
  if (rows > MOE_LINEAR_MAX_ROWS || columns > MOE_LINEAR_MAX_FEATURES) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scale) return MOE_ERR_NULL_PTR;
  if (ldx < columns || ldc < columns) return MOE_ERR_BAD_SHAPE;
  if (ldx > kFar || ldc > kFar || off(x, size_of(dtype)) || off(scale, 4)) return MOE_ERR_UNSUPPORTED;
  return quantise(dtype == MOE_DTYPE_F32, rows, columns, x, ldx, codes, ldc, columns, scale, PackItem{}, static_cast<hipStream_t>(stream));
}

int moe_linear_i8_workspace_size(const moe_linear_i8_config* cfg, int32_t max_rows, size_t* bytes) {
  const int st = check_i8(cfg, max_rows);
  if (st) return st;
  if (!bytes) return MOE_ERR_NULL_PTR;
  *bytes = i8_workspace(*cfg, max_rows);
  return MOE_OK;
}

int moe_linear_i8(const moe_linear_i8_config* cfg, int32_t M, const void* x, int64_t ldx, const float* x_scale,
                  const int8_t* w, int64_t ldw, const float* w_scale, const void* bias, const void* residual,
                  int64_t ldr, void* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_i8(cfg, M);
  if (st) return st;
  if (M == 0) return MOE_OK;
  const moe_linear_i8_config& c = *cfg;
  const bool codes = c.in_dtype == MOE_DTYPE_I8;
  if (!x || !w || !w_scale || !y || !workspace || (codes && !x_scale)) return MOE_ERR_NULL_PTR;
  const int N = c.out_features, K = c.in_features;
  if (ldx < K || ldw < K || ldy < N || (residual && ldr < N)) return MOE_ERR_BAD_SHAPE;
  if (ldx > kFar || ldw > kFar || ldy > kFar || (residual && ldr > kFar)) return MOE_ERR_UNSUPPORTED;
  if (residual == y && ldr != ldy) return MOE_ERR_BAD_SHAPE;
  if (workspace_bytes < i8_workspace(c, M)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (off(x, size_of(c.in_dtype)) || off(x_scale, 4) || off(w_scale, 4) || off(bias, size_of(c.bias_dtype)) ||
      off(residual, size_of(c.out_dtype)) || off(y, size_of(c.out_dtype)) || off(workspace, 16))
    return MOE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  Product g{{x, nullptr, ldx, 0, 0}, {w, nullptr, ldw, 0, 0}, M, N, K};
  const float* sx = x_scale;
  int8_t* q = static_cast<int8_t*>(workspace) + part_bytes(false, M, N);
  float* qs = reinterpret_cast<float*>(q + codes_bytes(c, M));
  const int64_t ld = codes_ld(c);
  const bool bf = c.bias_dtype == MOE_DTYPE_F32;
  const int row = static_cast<int>(align_up(K, 128));
  if (!codes && M == 1 && N <= kOnTheWayColumns && row <= kOnTheWayBytes && ldw < (int64_t{1} << 24)) {
    const bool aligned = aligned16(g.b, El::I8, true, N, K);
    const auto run = [&](auto rows, auto epi) { return launch_skinny<El::I8, false>(g, epi, aligned, part, s, rows, row + 16); };
    const auto with = [&](auto epi) {
      return c.in_dtype == MOE_DTYPE_F32 ? run(QuantisedRow<true>{x, qs, row}, epi) : run(QuantisedRow<false>{x, qs, row}, epi);
    };
    return c.out_dtype == MOE_DTYPE_F32 ? with(I8Out<true>{qs, w_scale, bias, residual, y, ldr, ldy, N, c.activation, bf})
                                        : with(I8Out<false>{qs, w_scale, bias, residual, y, ldr, ldy, N, c.activation, bf});
  }
  // What lies odd is laid out afresh; with values to quantise, in the quantiser's launch.
  PackArgs p{};
  if (large(c, M)) {
    if (codes && (K % 16 || ldx % 16 || off(x, 16))) {
      p.item[p.n++] = PackItem{x, q, ldx, ld, M, K, M};
      g.a.p = q;
      g.a.ld = ld;
    }
    if (K % 16) {
      int8_t* wq = reinterpret_cast<int8_t*>(qs) + align_up(static_cast<size_t>(M) * 4, 256);
      p.item[p.n++] = PackItem{w, wq, ldw, ld, N, K, N};
      g.b.p = wq;
      g.b.ld = ld;
      g.K = static_cast<int>(align_up(K, 16));
    }
  }
  if (!codes) {
    const int bad = quantise(c.in_dtype == MOE_DTYPE_F32, M, K, x, ldx, q, ld, static_cast<int>(ld), qs, p.item[0], s);
    if (bad) return bad;
    g.a.p = q;
    g.a.ld = ld;
    sx = qs;
  } else if (p.n && !pack_rows<uint8_t>(p, s)) {
    return MOE_ERR_LAUNCH_FAILED;
  }
  if (c.out_dtype == MOE_DTYPE_F32)
    return run_product<El::I8, true, true, false>(g, I8Out<true>{sx, w_scale, bias, residual, y, ldr, ldy, N, c.activation, bf}, part, s);
  return run_product<El::I8, true, true, false>(g, I8Out<false>{sx, w_scale, bias, residual, y, ldr, ldy, N, c.activation, bf}, part, s);
}

}  // extern "C"
