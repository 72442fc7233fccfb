// Dense matrix product with its epilogue: y = act(x W^T + bias) + residual.
//
// Sums run in float32 over the whole contraction; bias, activation and residual are
// applied to the float32 sum, which is rounded once, to y's type.
#include <algorithm>

#include "moe_mi355x.h"
#include "schedule.h"

namespace moe {
namespace {

struct LinearArgs {
  const void *x, *w, *bias, *residual;
  void* y;
  int64_t ldx, ldw, ldr, ldy;    // elements
  int M, N, K;
  int act;
};

// ---------------------------------------------------------------- epilogue

// tanh(u) = 1 - 2 / (1 + e^(2u)): exact at both infinities, and near 0 within a few
// 2^-24 of 1, which is what the 1 + tanh of the activation keeps of it.
__device__ __forceinline__ float tanh_f32(float u) { return 1.0f - 2.0f / (1.0f + expf(2.0f * u)); }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_RELU: return v < 0.0f ? 0.0f : v;                              // NaN stays NaN
    case MOE_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678f));
    case MOE_ACT_GELU_TANH: return 0.5f * v * (1.0f + tanh_f32(0.79788456f * (v + 0.044715f * v * v * v)));
    case MOE_ACT_SILU: return v / (1.0f + expf(-v));
    default: return v;
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
  if (a.bias) v += elem<F32>(a.bias, n);
  v = activate(v, a.act);
  if (a.residual) v += elem<OUT32>(a.residual, static_cast<size_t>(m) * a.ldr + n);
  const size_t o = static_cast<size_t>(m) * a.ldy + n;
  if constexpr (OUT32) static_cast<float*>(a.y)[o] = v;
  else static_cast<uint16_t*>(a.y)[o] = f32_to_bf16_bits(v);
}

// ---------------------------------------------------------------- any size and alignment
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

size_t linear_workspace(const moe_linear_config&, int32_t) { return 256; }

bool off(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == MOE_DTYPE_F32 ? 4 : 2) != 0; }

template <bool F32, bool OUT32>
int linear_launch(const LinearArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(a.N, kAnyTile)), static_cast<unsigned>(ceil_div(a.M, kAnyTile)));
  linear_any_kernel<F32, OUT32><<<grid, 256, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
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
  if (cfg->in_dtype == MOE_DTYPE_F32) return linear_launch<true, true>(a, s);
  return cfg->out_dtype == MOE_DTYPE_F32 ? linear_launch<false, true>(a, s) : linear_launch<false, false>(a, s);
}

}  // extern "C"
