// The norms before and after a block, with the block's gate and the residual's scale:
//   z = a r + b gate * post(y),  out = norm(z)
// where norm(v) = n(v) w + bias, n(v) = v / sqrt(mean(v^2) + eps), or of v - mean(v), and
// post is such a norm with its own weight, or nothing.  All in float32 from the loaded
// elements on; z and out are rounded once (out comes from the unrounded z).
//
// Backward, from dz and dout, for the stored z:
//   dn = dout w,  zt = dz + (dn - n(z) mean(dn n(z)) [- mean(dn)]) / dev(z)
//   dr = a zt,  dv = b gate zt,  dgate = b zt post(y),  dy = dv through post likewise
//   dw = sum over rows of dout n(z), ...
// Statistics are taken again from y and z, whose rows are in registers anyway, so nothing
// has to be kept between the passes but z.  The sums over rows stay in registers over all
// rows of a workgroup; a second launch adds the workgroups' sums in order.
//
// A row belongs to as many waves as give each lane C times eight of its elements; a wave
// that holds a whole row needs no barrier.
//
// Bound by memory, or for few rows by one launch: 8192 x 7168 in bf16 with a post norm takes
// 94 to 100 us (4.9 TB/s over four tensors, what a large copy reaches), one row 3 us on the
// GPU.  Backward, six tensors and three sums over rows, 150 to 158 (4.6 TB/s), of which 9 are
// the second launch's.  (Call after call, from the second hundred on; the first hundred after
// a pause take up to a tenth longer.)  With f32 throughout 176 and 332.  Rows wider than 8192
// run as fast forward (8192 x 12288 169 us), but not backward: 2.0 ms (norm_back.h).
#include <algorithm>
#include <initializer_list>

#include "norm_back.h"

namespace moe {
namespace {

struct NormArgs {
  const void *y, *r, *gate, *w, *wb, *pw, *pb;
  void *z, *out;
  float* out_scale;
  int64_t ldy, ldr, ldg, ldz, ldo;
  int T, H, waves;
  float eps, a, b;
  int layer, gate_kind, params_f32, out_dtype;
};

// mean (layer norms) and 1 / deviation of the C x 8 elements of each lane.
template <int C>
__device__ __forceinline__ void statistics(const float (&v)[C][8], const NormArgs& a, int at, int width, int wave,
                                           RowLds<float>& lds, int& turn, float& mean, float& rstd) {
  float s[1] = {0.0f};
  mean = 0.0f;
  if (a.layer) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[c][e];           // zeros behind the row's end
    row_all(s, wave, a.waves, lds, turn, Add{});
    mean = s[0] / a.H;
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Columns col(c, at, width, a.H);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < col.left ? v[c][e] - mean : 0.0f;
        s[0] = fmaf(d, d, s[0]);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(v[c][e], v[c][e], s[0]);
  }
  row_all(s, wave, a.waves, lds, turn, Add{});
  rstd = 1.0f / sqrtf(s[0] / a.H + a.eps);
}

template <bool YF32, bool SF32, int C>
__global__ void __launch_bounds__(C == 1 ? 1024 : 512) norm_kernel(NormArgs a) {
  __shared__ RowLds<float> lds;
  __shared__ RowLds<uint32_t> lds_bits;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Rows of one wave come several to a workgroup.
  const int in_row = a.waves > 1 ? wave : 0;
  const int64_t t = a.waves > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + wave;
  if (t >= a.T) return;
  const int at = in_row * 64 + lane, width = a.waves * 64;
  int turn = 0;
  const bool pf = a.params_f32;
  Raw8<YF32> yr[C];
  Raw8<SF32> rr[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Columns col(c, at, width, a.H);
    yr[c] = load8<YF32>(static_cast<const uint8_t*>(a.y) + t * a.ldy * (YF32 ? 4 : 2), col.i, col.left);
  }
  if (a.r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Columns col(c, at, width, a.H);
      rr[c] = load8<SF32>(static_cast<const uint8_t*>(a.r) + t * a.ldr * (SF32 ? 4 : 2), col.i, col.left);
    }
  }
  const float gate_token = a.gate_kind == MOE_GATE_TOKEN ? load_of(pf, a.gate, t) : 1.0f;
  // With one chunk the parameters are in flight beside the row; with more they are read
  // where they are used.
  float w8[8], wb8[8], pw8[8], pb8[8], g8[8];
  const auto param = [&](const void* p, int c, float (&v)[8]) {
    const Columns col(c, at, width, a.H);
    load8_of(pf, p, col.i, col.left, v);
  };
  const void* gate_row = a.gate_kind == MOE_GATE_FULL ? static_cast<const uint8_t*>(a.gate) + t * a.ldg * (pf ? 4 : 2) : a.gate;
  const bool gate_columns = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL;
  if constexpr (C == 1) {
    if (a.w) param(a.w, 0, w8);
    if (a.wb) param(a.wb, 0, wb8);
    if (a.pw) param(a.pw, 0, pw8);
    if (a.pb) param(a.pb, 0, pb8);
    if (gate_columns) param(gate_row, 0, g8);
  }
  float v[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = value<YF32>(yr[c], e);
  float mean, rstd;
  if (a.pw) {
    statistics(v, a, at, width, in_row, lds, turn, mean, rstd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (C > 1) param(a.pw, c, pw8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = (v[c][e] - mean) * rstd * pw8[e];
      if (a.pb) {
        if constexpr (C > 1) param(a.pb, c, pb8);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] += pb8[e];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Columns col(c, at, width, a.H);
    if (gate_columns) {
      if constexpr (C > 1) param(gate_row, c, g8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= g8[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= gate_token;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = a.r ? a.a * value<SF32>(rr[c], e) + a.b * v[c][e] : a.b * v[c][e];
    // Nothing but zeros behind the row's end, whatever is in the scales.
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = e < col.left ? v[c][e] : 0.0f;
    if (a.z) store8<SF32>(a.z, t * a.ldz + col.i, v[c], col.left);
  }
  if (!a.out) return;
  statistics(v, a, at, width, in_row, lds, turn, mean, rstd);
  uint32_t most[1] = {0};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Columns col(c, at, width, a.H);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] = (v[c][e] - mean) * rstd;
    if (a.w) {
      if constexpr (C > 1) param(a.w, c, w8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= w8[e];
    }
    if (a.wb) {
      if constexpr (C > 1) param(a.wb, c, wb8);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] += wb8[e];
    }
    if (a.out_dtype == MOE_DTYPE_I8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < col.left) most[0] = max(most[0], __float_as_uint(v[c][e]) & 0x7fffffffu);
    } else if (a.out_dtype == MOE_DTYPE_F32) {
      store8<true>(a.out, t * a.ldo + col.i, v[c], col.left);
    } else {
      store8<false>(a.out, t * a.ldo + col.i, v[c], col.left);
    }
  }
  if (a.out_dtype != MOE_DTYPE_I8) return;
  int turn_bits = 0;
  row_all(most, in_row, a.waves, lds_bits, turn_bits, Most{});
  const float s = i8_scale(most[0]), inv = 1.0f / s;
  if (at == 0) a.out_scale[t] = s;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const Columns col(c, at, width, a.H);
    store_codes(static_cast<int8_t*>(a.out) + t * a.ldo + col.i, v[c], s, inv, col.left);
  }
}

// ---------------------------------------------------------------- sums over rows

// The groups' sums added in order: 16 columns to a workgroup, the groups in 64 ranges.
struct NormSums {
  void* out[kSums];
  const float* part;
  int H, groups, n, f32;
};
__global__ void __launch_bounds__(1024) norm_sums_kernel(NormSums a) {
  __shared__ float red[64][16];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4, k = blockIdx.y, col = blockIdx.x * 16 + c;
  const int lo = q * a.groups / 64, hi = (q + 1) * a.groups / 64;
  float s = 0.0f;
  if (col < a.H) {
    const float* p = a.part + static_cast<size_t>(k) * a.H + col;
    const size_t step = static_cast<size_t>(a.n) * a.H;
    constexpr int kAhead = 8;
    for (int g = lo; g < hi; g += kAhead) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = g + i < hi ? p[(g + i) * step] : 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s += v[i];
    }
  }
  red[q][c] = s;
  __syncthreads();
  if (q >= 4) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += red[16 * q + i][c];
  // The four ranges' lanes of a column are 16 apart in one wave.
  s += __shfl_xor(s, 16, kWave);
  s += __shfl_xor(s, 32, kWave);
  if (q == 0 && col < a.H) store_of(a.f32, a.out[k], col, s);
}

// ---------------------------------------------------------------- host

bool plain_type(int d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16; }
size_t type_size(int d) { return d == MOE_DTYPE_F32 ? 4 : d == MOE_DTYPE_BF16 ? 2 : 1; }

int check_norm(const moe_norm_config* c, int32_t rows) {
  if (!c) return MOE_ERR_NULL_PTR;
  if (!plain_type(c->block_dtype) || !plain_type(c->stream_dtype) || !plain_type(c->param_dtype) ||
      !(plain_type(c->out_dtype) || c->out_dtype == MOE_DTYPE_I8))
    return MOE_ERR_BAD_DTYPE;
  if (c->hidden_size <= 0 || rows < 0) return MOE_ERR_BAD_SHAPE;
  if (c->kind != MOE_NORM_RMS && c->kind != MOE_NORM_LAYER) return MOE_ERR_BAD_SHAPE;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_FULL) return MOE_ERR_BAD_SHAPE;
  if (!(c->eps >= 0.0f)) return MOE_ERR_BAD_SHAPE;
  if (c->hidden_size > MOE_NORM_MAX_HIDDEN || rows > MOE_LINEAR_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A matrix operand: its stride and its alignment.
int check_rows(const void* p, int64_t ld, int64_t width, size_t size) {
  if (!p) return MOE_OK;
  if (ld < width) return MOE_ERR_BAD_SHAPE;
  if (ld > (int64_t{1} << 40) || reinterpret_cast<uintptr_t>(p) % size) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
int first(std::initializer_list<int> st) {
  for (int s : st)
    if (s) return s;
  return MOE_OK;
}

// Chunks of eight elements to a lane and waves to a row.
struct RowPlan {
  int chunks, waves;
};
RowPlan row_plan(int H, int max_waves_of_one) {
  const int lanes = static_cast<int>(ceil_div(H, 8));
  for (int c : {1, 2, 4}) {
    const int waves = static_cast<int>(ceil_div(lanes, 64 * c));
    if (waves <= (c == 1 ? max_waves_of_one : 8)) return {c, waves};
  }
  return {4, 8};
}

template <bool YF32, bool SF32>
int launch_norm(const NormArgs& a, int chunks, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.waves > 1 ? a.T : ceil_div(a.T, kRowsOfOneWave));
  const unsigned block = 64u * static_cast<unsigned>(a.waves > 1 ? a.waves : kRowsOfOneWave);
  if (chunks == 1) norm_kernel<YF32, SF32, 1><<<grid, block, 0, s>>>(a);
  else if (chunks == 2) norm_kernel<YF32, SF32, 2><<<grid, block, 0, s>>>(a);
  else norm_kernel<YF32, SF32, 4><<<grid, block, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
}

// Groups of rows of a backward pass.  A group is a workgroup, as many to a CU as make 16 waves,
// or for rows of up to 512 columns one wave, eight to a CU (two workgroups of four).  Of few
// rows there are fewer groups: as many as rows up to 256, then 256 until a group has eight rows
// (four where it is one wave), and with those up to the CUs' fill.
int norm_groups(const moe_norm_config& c, int64_t T) {
  const int waves = static_cast<int>(ceil_div(c.hidden_size, 512));
  const int64_t most = waves == 1 ? 256 * 4 * 2 : 256 * std::max(1, 16 / waves);
  // A group of few rows writes nearly as much as it reads: 1001 x 1537 with five sums takes
  // 43 us with one row to a group, 25 with two or four.
  const int64_t rows = waves == 1 ? 4 : 8;
  return static_cast<int>(std::min({T, most, std::max<int64_t>(256, T / rows)}));
}
size_t norm_back_bytes(const moe_norm_config& c, int64_t T) {
  return std::max<size_t>(static_cast<size_t>(norm_groups(c, T)) * kSums * c.hidden_size * sizeof(float), 256);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm(const moe_norm_config* cfg, int32_t T, const void* y, int64_t ldy, const void* residual, int64_t ldr,
             const void* gate, int64_t ldg, const void* weight, const void* bias, const void* post_weight,
             const void* post_bias, void* z, int64_t ldz, void* out, int64_t ldo, float* out_scale, void* stream) {
  const int st = check_norm(cfg, T);
  if (st) return st;
  if (T == 0) return MOE_OK;
  const moe_norm_config& c = *cfg;
  if (!y || (!z && !out) || (c.gate != MOE_GATE_NONE && !gate)) return MOE_ERR_NULL_PTR;
  if ((post_bias && !post_weight) || (out && c.out_dtype == MOE_DTYPE_I8 && !out_scale)) return MOE_ERR_NULL_PTR;
  const int64_t H = c.hidden_size;
  const size_t ps = type_size(c.param_dtype), ss = type_size(c.stream_dtype);
  const int bad = first({check_rows(y, ldy, H, type_size(c.block_dtype)), check_rows(residual, ldr, H, ss),
                         c.gate == MOE_GATE_FULL ? check_rows(gate, ldg, H, ps) : check_rows(gate, H, H, ps),
                         check_rows(weight, H, H, ps), check_rows(bias, H, H, ps), check_rows(post_weight, H, H, ps),
                         check_rows(post_bias, H, H, ps), check_rows(z, ldz, H, ss),
                         check_rows(out, ldo, H, type_size(c.out_dtype)), check_rows(out_scale, 1, 1, 4)});
  if (bad) return bad;
  if (z && z == residual && ldz != ldr) return MOE_ERR_BAD_SHAPE;
  // Few rows: as many lanes as there are, for the latency.  Many: several chunks to a lane,
  // for the loads in flight.  Microseconds of the first and the second (with a post norm):
  // 16 x 5120 4.0 and 4.5, 256 x 7168 5.4 and 5.6, 512 x 7168 8.9 and 8.0, 4096 x 7168 57 and 40.
  const RowPlan p = row_plan(c.hidden_size, T <= 256 ? 16 : 2);
  NormArgs a{};
  a.y = y, a.r = residual, a.gate = c.gate == MOE_GATE_NONE ? nullptr : gate, a.w = weight, a.wb = bias;
  a.pw = post_weight, a.pb = post_bias, a.z = z, a.out = out, a.out_scale = out_scale;
  a.ldy = ldy, a.ldr = ldr, a.ldg = ldg, a.ldz = ldz, a.ldo = ldo;
  a.T = T, a.H = c.hidden_size, a.waves = p.waves;
  a.eps = c.eps, a.a = c.residual_scale, a.b = c.block_scale;
  a.layer = c.kind == MOE_NORM_LAYER, a.gate_kind = c.gate, a.params_f32 = c.param_dtype == MOE_DTYPE_F32;
  a.out_dtype = c.out_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool yf = c.block_dtype == MOE_DTYPE_F32, sf = c.stream_dtype == MOE_DTYPE_F32;
  if (yf) return sf ? launch_norm<true, true>(a, p.chunks, s) : launch_norm<true, false>(a, p.chunks, s);
  return sf ? launch_norm<false, true>(a, p.chunks, s) : launch_norm<false, false>(a, p.chunks, s);
}

int moe_norm_backward_workspace_size(const moe_norm_config* cfg, int32_t max_rows, size_t* bytes) {
  const int st = check_norm(cfg, max_rows);
  if (st) return st;
  if (!bytes) return MOE_ERR_NULL_PTR;
  *bytes = norm_back_bytes(*cfg, max_rows);
  return MOE_OK;
}

int moe_norm_backward(const moe_norm_config* cfg, int32_t T, const void* y, int64_t ldy, const void* z, int64_t ldz,
                      const void* gate, int64_t ldg, const void* weight, const void* post_weight,
                      const void* post_bias, const void* dz, int64_t lddz, const void* dout, int64_t lddo, void* dy,
                      int64_t lddy, void* dresidual, int64_t lddr, void* dgate, int64_t lddg, void* dweight,
                      void* dbias, void* dpost_weight, void* dpost_bias, void* workspace, size_t workspace_bytes,
                      void* stream) {
  const int st = check_norm(cfg, T);
  if (st) return st;
  const moe_norm_config& c = *cfg;
  if (c.out_dtype == MOE_DTYPE_I8) return MOE_ERR_BAD_DTYPE;
  if (dgate && c.gate == MOE_GATE_NONE) return MOE_ERR_BAD_SHAPE;
  const int64_t H = c.hidden_size;
  const size_t ps = type_size(c.param_dtype), ss = type_size(c.stream_dtype), bs = type_size(c.block_dtype);
  int bad = first({check_rows(dweight, H, H, ps), check_rows(dbias, H, H, ps), check_rows(dpost_weight, H, H, ps),
                   check_rows(dpost_bias, H, H, ps), check_rows(dgate, c.gate == MOE_GATE_FULL ? lddg : H, H, ps)});
  if (bad) return bad;
  if (T > 0) {
    if (!y || !workspace || (!dz && !dout) || (dout && !z) || (c.gate != MOE_GATE_NONE && !gate)) return MOE_ERR_NULL_PTR;
    if ((dweight || dbias) && !dout) return MOE_ERR_NULL_PTR;
    if ((post_bias || dpost_weight || dpost_bias) && !post_weight) return MOE_ERR_NULL_PTR;
    bad = first({check_rows(y, ldy, H, bs), check_rows(z, ldz, H, ss),
                 check_rows(gate, c.gate == MOE_GATE_FULL ? ldg : H, H, ps), check_rows(weight, H, H, ps),
                 check_rows(post_weight, H, H, ps), check_rows(post_bias, H, H, ps), check_rows(dz, lddz, H, ss),
                 check_rows(dout, lddo, H, type_size(c.out_dtype)), check_rows(dy, lddy, H, bs),
                 check_rows(dresidual, lddr, H, ss), check_rows(workspace, 1, 1, 16)});
    if (bad) return bad;
    if (dz && dz == dresidual && lddz != lddr) return MOE_ERR_BAD_SHAPE;
    if (workspace_bytes < norm_back_bytes(c, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  NormBackArgs a{};
  a.y = y, a.z = z, a.gate = c.gate == MOE_GATE_NONE ? nullptr : gate, a.w = weight, a.pw = post_weight, a.pb = post_bias;
  a.dz = dz, a.dout = dout, a.dy = dy, a.dr = dresidual, a.dgate = dgate, a.part = static_cast<float*>(workspace);
  a.ldy = ldy, a.ldz = ldz, a.ldg = ldg, a.lddz = lddz, a.lddo = lddo, a.lddy = lddy, a.lddr = lddr, a.lddg = lddg;
  a.T = T, a.H = c.hidden_size, a.groups = norm_groups(c, T);
  a.eps = c.eps, a.a = c.residual_scale, a.b = c.block_scale;
  a.layer = c.kind == MOE_NORM_LAYER, a.gate_kind = c.gate;
  NormSums sums{};
  void* outs[kSums] = {dweight, dbias, dpost_weight, dpost_bias, c.gate == MOE_GATE_CHANNEL ? dgate : nullptr};
  for (int i = 0; i < kSums; ++i)
    if (outs[i]) {
      a.sums |= 1 << i;
      sums.out[sums.n++] = outs[i];
    }
  sums.part = a.part, sums.H = c.hidden_size, sums.groups = a.groups, sums.f32 = c.param_dtype == MOE_DTYPE_F32;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T > 0) {
    const bool sf = c.stream_dtype == MOE_DTYPE_F32, of = c.out_dtype == MOE_DTYPE_F32, pf = c.param_dtype == MOE_DTYPE_F32;
    const bool bias = dbias || dpost_bias || post_bias;
    if (c.block_dtype == MOE_DTYPE_F32) launch_norm_back_f32(a, s, sf, of, pf, bias);
    else launch_norm_back_bf16(a, s, sf, of, pf, bias);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  }
  if (sums.n) {
    norm_sums_kernel<<<dim3(static_cast<unsigned>(ceil_div(H, 16)), static_cast<unsigned>(sums.n)), 1024, 0, s>>>(sums);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  }
  return MOE_OK;
}

}  // extern "C"
