// The backward pass of the norms (norm.hip has its mathematics), compiled for either type of
// the block's output.
#pragma once

#include <type_traits>

#include "moe_mi355x.h"
#include "rows.h"

namespace moe {

struct NormBackArgs {
  const void *y, *z, *gate, *w, *pw, *pb, *dz, *dout;
  void *dy, *dr, *dgate;
  float* part;                       // [groups][sums][H]
  int64_t ldy, ldz, ldg, lddz, lddo, lddy, lddr, lddg;
  int T, H, waves, groups;           // waves of a row: the launch sets them
  float eps, a, b;
  int layer, gate_kind;
  int sums;                          // bits of Sum
};
// The sums over rows, in the order in which a group stores them.
enum Sum { kSumW = 1, kSumWb = 2, kSumPw = 4, kSumPb = 8, kSumGate = 16 };
constexpr int kSums = 5;

constexpr int kRowsOfOneWave = 4;      // to a workgroup, where a row is one wave's

// Launch on a stream; flags: whether stream, out and parameters are float32, and whether
// there are biases or their gradients.
void launch_norm_back_f32(const NormBackArgs& a, hipStream_t s, bool sf, bool of, bool pf, bool bias);
void launch_norm_back_bf16(const NormBackArgs& a, hipStream_t s, bool sf, bool of, bool pf, bool bias);

namespace {

// Eight columns of a row: chunk c of lane `at`, of a row's `width` lanes.
struct Columns {
  int i, left;
  __device__ __forceinline__ Columns(int c, int at, int width, int H) : i(8 * (at + c * width)), left(H - i) {}
};

#ifdef MOE_NORM_BACK_KERNELS

// BIAS: with sums for biases.  A workgroup's parameters and sums stay over its rows, and the
// next row's loads are in flight while a row is worked on: in registers, where they fit.
//
// Most waves to a row: with one chunk to a lane everything in bf16 takes 121 registers, the
// other forms up to 168, and none uses scratch memory.  Two chunks take 218 to 256; with biases
// all of these spill (72 to 256 bytes a lane), without them 4 of 16 do (up to 76).  Four
// chunks, of rows wider than 8192, spill 1256 to 1620 bytes a lane and are bound by that:
// bf16 8192 x 12288 takes 2.0 ms, 8192 x 16384 2.9, where the rows alone are 0.25 and 0.33.
// 8192 x 5120 took 127 us in ten waves of one chunk and 164 in five of two, measured in turn (117 in
// ten since); bf16 8192 x 7168 layer norms with biases, in two chunks, take 262, rms norms
// without, in one, 153.
constexpr int back_waves(bool narrow, int chunks) { return chunks > 1 ? 8 : narrow ? 16 : 12; }

template <bool YF32, bool SF32, bool OF32, bool PF32, bool BIAS, int C>
__global__ void __launch_bounds__(64 * back_waves(!YF32 && !SF32 && !OF32 && !PF32 && !BIAS, C)) norm_back_kernel(NormBackArgs a) {
  __shared__ RowLds<float> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int in_row = a.waves > 1 ? wave : 0;
  const int group = a.waves > 1 ? blockIdx.x : static_cast<int>(blockIdx.x) * (blockDim.x >> 6) + wave;
  if (group >= a.groups) return;
  const int at = in_row * 64 + lane, width = a.waves * 64;
  int turn = 0;
  const float inv_h = 1.0f / a.H;
  float sum_w[C][8], sum_pw[C][8], sum_g[C][8], sum_wb[BIAS ? C : 1][8], sum_pb[BIAS ? C : 1][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sum_w[c][e] = sum_pw[c][e] = sum_g[c][e] = 0.0f;
      if constexpr (BIAS) sum_wb[c][e] = sum_pb[c][e] = 0.0f;
    }
  struct Row {
    Raw8<YF32> y[C];
    Raw8<SF32> z[C], dz[C];
    Raw8<OF32> dout[C];
    float token;
  };
  const bool post = a.pw, weighted = a.w && a.dout;
  const bool need_y = post || (a.gate_kind != MOE_GATE_NONE && a.dgate);
  const auto rows = [&](auto f32, const void* p, int64_t ld, int64_t t, int c) __attribute__((always_inline)) {
    const Columns col(c, at, width, a.H);
    return load8<decltype(f32)::value>(static_cast<const uint8_t*>(p) + t * ld * (decltype(f32)::value ? 4 : 2), col.i, col.left);
  };
  const auto load = [&](Row& R, int64_t t) __attribute__((always_inline)) {
    R.token = a.gate_kind == MOE_GATE_TOKEN ? load_of(PF32, a.gate, t) : 1.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (need_y) R.y[c] = rows(std::bool_constant<YF32>{}, a.y, a.ldy, t, c);
      if (a.dz) R.dz[c] = rows(std::bool_constant<SF32>{}, a.dz, a.lddz, t, c);
      if (a.dout) {
        R.z[c] = rows(std::bool_constant<SF32>{}, a.z, a.ldz, t, c);
        R.dout[c] = rows(std::bool_constant<OF32>{}, a.dout, a.lddo, t, c);
      }
    }
  };
  Row R;
  load(R, group);
  // The parameters; ones for what is not there.
  const uint32_t one = PF32 ? 0x3f800000u : 0x3f803f80u;
  Raw8<PF32> w[C], pw[C], g[C], pb[BIAS ? C : 1];
  const bool by_channel = a.gate_kind == MOE_GATE_CHANNEL, by_element = a.gate_kind == MOE_GATE_FULL;
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int k = 0; k < (PF32 ? 2 : 1); ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[c].v[k][e] = pw[c].v[k][e] = g[c].v[k][e] = one;
    if (weighted) w[c] = rows(std::bool_constant<PF32>{}, a.w, 0, 0, c);
    if (post) pw[c] = rows(std::bool_constant<PF32>{}, a.pw, 0, 0, c);
    if (by_channel) g[c] = rows(std::bool_constant<PF32>{}, a.gate, 0, 0, c);
    if constexpr (BIAS)
      if (a.pb) pb[c] = rows(std::bool_constant<PF32>{}, a.pb, 0, 0, c);
  }
  for (int64_t t = group; t < a.T; t += a.groups) {
    float y[C][8], z[C][8], zt[C][8], dn[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[c][e] = need_y ? value<YF32>(R.y[c], e) : 0.0f;
        zt[c][e] = a.dz ? value<SF32>(R.dz[c], e) : 0.0f;
        z[c][e] = a.dout ? value<SF32>(R.z[c], e) : 0.0f;
        dn[c][e] = a.dout ? value<OF32>(R.dout[c], e) : 0.0f;
      }
    const float gate_token = R.token;
    if (by_element) {
#pragma unroll
      for (int c = 0; c < C; ++c) g[c] = rows(std::bool_constant<PF32>{}, a.gate, a.ldg, t, c);
    }
    // (Nothing behind the group's last row: another one's dz may be dresidual's place, which its
    // own group is writing.)
    if (t + a.groups < a.T) load(R, t + a.groups);

    // Statistics of z and y, and z's sums with dn.
    float zmean = 0.0f, ymean = 0.0f;
    if (a.layer) {
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] += z[c][e];
          s[1] += y[c][e];
        }
      row_all(s, in_row, a.waves, lds, turn, Add{});
      zmean = s[0] * inv_h;
      ymean = post ? s[1] * inv_h : 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Columns col(c, at, width, a.H);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z[c][e] = e < col.left ? z[c][e] - zmean : 0.0f;
          y[c][e] = e < col.left ? y[c][e] - ymean : 0.0f;
        }
      }
    }
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = dn[c][e] * value<PF32>(w[c], e);
        s[0] = fmaf(z[c][e], z[c][e], s[0]);
        s[1] = fmaf(d, z[c][e], s[1]);
        s[2] = fmaf(y[c][e], y[c][e], s[2]);
        s[3] += d;
      }
    row_all(s, in_row, a.waves, lds, turn, Add{});
    const float zr = 1.0f / sqrtf(s[0] * inv_h + a.eps), yr = post ? 1.0f / sqrtf(s[2] * inv_h + a.eps) : 1.0f;
    const float m = s[1] * inv_h * zr, dmean = a.layer ? s[3] * inv_h : 0.0f;
    // zt and dr; y becomes n(y), dn the gradient of n(y).
    float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Columns col(c, at, width, a.H);
      float t8[8];
      if (a.dout) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = z[c][e] * zr;
          sum_w[c][e] = fmaf(dn[c][e], n, sum_w[c][e]);
          if constexpr (BIAS) sum_wb[c][e] += dn[c][e];
          zt[c][e] = fmaf(zr, dn[c][e] * value<PF32>(w[c], e) - fmaf(n, m, dmean), zt[c][e]);
        }
      }
      if (a.dr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t8[e] = a.a * zt[c][e];
        store8<SF32>(a.dr, t * a.lddr + col.i, t8, col.left);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = y[c][e] * yr, p = value<PF32>(pw[c], e);
        float v = n * p;
        if constexpr (BIAS) v += a.pb ? value<PF32>(pb[c], e) : 0.0f;
        const float dv0 = e < col.left ? a.b * zt[c][e] : 0.0f;
        t8[e] = dv0 * v;
        sum_g[c][e] += t8[e];
        q[2] += t8[e];
        const float dv = dv0 * value<PF32>(g[c], e) * gate_token;
        sum_pw[c][e] = fmaf(dv, n, sum_pw[c][e]);
        if constexpr (BIAS) sum_pb[c][e] += dv;
        const float dp = dv * p;
        q[0] = fmaf(dp, n, q[0]);
        q[1] += dp;
        y[c][e] = n;
        dn[c][e] = dp;
      }
      if (by_element && a.dgate) store8<PF32>(a.dgate, t * a.lddg + col.i, t8, col.left);
    }
    const bool by_token = a.gate_kind == MOE_GATE_TOKEN && a.dgate;
    if (post || by_token) row_all(q, in_row, a.waves, lds, turn, Add{});
    if (by_token && at == 0) store_of(PF32, a.dgate, t, q[2]);
    if (a.dy) {
      const float pm = q[0] * inv_h, pd = a.layer ? q[1] * inv_h : 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Columns col(c, at, width, a.H);
        if (post) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dn[c][e] = yr * (dn[c][e] - fmaf(y[c][e], pm, pd));
        }
        store8<YF32>(a.dy, t * a.lddy + col.i, dn[c], col.left);
      }
    }
  }
  int k = 0;
  const auto out = [&](int bit, const auto& sum) __attribute__((always_inline)) {
    if (!(a.sums & bit)) return;
    float* p = a.part + (static_cast<size_t>(group) * __popc(a.sums) + k++) * a.H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const Columns col(c, at, width, a.H);
      store8<true>(p, col.i, sum[c], col.left);
    }
  };
  out(kSumW, sum_w);
  if constexpr (BIAS) out(kSumWb, sum_wb);
  out(kSumPw, sum_pw);
  if constexpr (BIAS) out(kSumPb, sum_pb);
  out(kSumGate, sum_g);
}

template <bool YF32, bool SF32, bool OF32, bool PF32, bool BIAS>
void launch_norm_back(NormBackArgs a, hipStream_t s) {
  const int lanes = static_cast<int>(ceil_div(a.H, 8));
  const int chunks = lanes <= 64 * back_waves(!YF32 && !SF32 && !OF32 && !PF32 && !BIAS, 1) ? 1 : lanes <= 1024 ? 2 : 4;
  a.waves = static_cast<int>(ceil_div(lanes, 64 * chunks));
  const unsigned grid = static_cast<unsigned>(a.waves > 1 ? a.groups : ceil_div(a.groups, kRowsOfOneWave));
  const unsigned block = 64u * static_cast<unsigned>(a.waves > 1 ? a.waves : kRowsOfOneWave);
  if (chunks == 1) norm_back_kernel<YF32, SF32, OF32, PF32, BIAS, 1><<<grid, block, 0, s>>>(a);
  else if (chunks == 2) norm_back_kernel<YF32, SF32, OF32, PF32, BIAS, 2><<<grid, block, 0, s>>>(a);
  else norm_back_kernel<YF32, SF32, OF32, PF32, true, 4><<<grid, block, 0, s>>>(a);
}
// One type after the other becomes a constant.
template <bool... KNOWN, class... REST>
void pick_norm_back(const NormBackArgs& a, hipStream_t s, bool next, REST... rest) {
  if constexpr (sizeof...(REST) == 0)
    next ? launch_norm_back<KNOWN..., true>(a, s) : launch_norm_back<KNOWN..., false>(a, s);
  else
    next ? pick_norm_back<KNOWN..., true>(a, s, rest...) : pick_norm_back<KNOWN..., false>(a, s, rest...);
}

#endif

}  // namespace
}  // namespace moe
