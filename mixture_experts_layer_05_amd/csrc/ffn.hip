// The dense gated FFN, y = (act(x Wg^T) * (x Wu^T)) Wd^T, and its gradients.
//
// Forward: one product computes g = x Wg^T and u = x Wu^T side by side (their columns
// take turns in a tile, so that a lane gets both of an element) and its epilogue writes
// h = act(g) u; the down projection is another product.  For a backward pass the
// epilogue also keeps a = act(g) and b = u act'(g), in float32.
//
// Backward, from dy:
//   dh = dy Wd,  du = dh a,  dg = dh b         one product, the two gradients its epilogue
//   dx = dg Wg + du Wu                         one product over both halves of [dg du]
//   dWg = dg^T x, dWu = du^T x                 one product of 2 I rows
//   dWd = dy^T h
// h, dg and du are matrix operands and have the weights' type: with bf16 weights each is
// rounded once.  (Of up to eight rows the forward pass keeps what h's rounding leaves as eight
// rows more, which a tile of 16 has free: y's own rounding is then the only one.)  a and b stay in float32: one more rounding of either would add to dg's
// and du's own (weight gradients off by 1.7 roundings instead of 1.4).
//
// Bound by memory up to 16 rows, by the matrix cores from about 500 on, in between by what
// a CU takes in and by the launches.  Weights of 5120 x 17408 in bf16: one row 104 us (three
// matrices at 5.1 TB/s), a training step of 8192 rows 10.6 to 11.3 ms for 13.1 TFLOP (1.16 to
// 1.24 PFLOP/s; the nine products alone take 12.1 ms in library calls).
#include "gemm.h"
#include "pack.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- epilogues

// act(v) and act'(v).
template <bool QUICK>
__device__ __forceinline__ void act_slope(float v, int act, float& f, float& d) {
  const auto sigmoid = [](float u) {
    if constexpr (QUICK) return __builtin_amdgcn_rcpf(1.0f + __expf(-u));
    else return 1.0f / (1.0f + expf(-u));
  };
  switch (act) {
    case MOE_ACT_RELU:
      f = v < 0.0f ? 0.0f : v;                    // NaN stays NaN
      d = v > 0.0f ? 1.0f : 0.0f;
      break;
    case MOE_ACT_GELU: {
      const float c = 0.5f * (1.0f + erff(v * 0.70710678f));
      f = v * c;
      d = c + (fabsf(v) < 40.0f ? v * 0.39894228f * expf(-0.5f * v * v) : 0.0f);
      break;
    }
    case MOE_ACT_GELU_TANH: {
      const float s = sigmoid(1.59576912f * (v + 0.044715f * v * v * v)), t = s * (1.0f - s);
      f = v * s;
      // s (1 - s) is 0 far out, where v^2 may be infinite.
      d = s + (t > 0.0f ? v * t * 1.59576912f * (1.0f + 0.134145f * v * v) : 0.0f);
      break;
    }
    case MOE_ACT_SILU: {
      const float s = sigmoid(v);
      f = v * s;
      d = s + f * (1.0f - s);
      break;
    }
    default:
      f = v;
      d = 1.0f;
      break;
  }
}

struct None {};

// h = act(g) u, what its rounding leaves (`rests`) eight rows on, and a and b where they are
// kept; their rows lie `ld`, a multiple of eight, apart, so that a whole quad may be written
// at their ends.  The eight elements that a row of h ends in are written, zeros behind its end.
template <bool F32, bool KEEP>
struct GatedOut {
  static constexpr int kAhead = 4;
  using Cols = None;
  using Ahead = None;
  void* h;
  float *a, *b;
  int64_t ld;
  int N, act;
  bool rests;
  // (Without a and b: the tiles, and with them the sums' order and y's bits, are the same
  // whether they are kept or not.)
  int bytes() const { return F32 ? 4 : 2; }
  __device__ __forceinline__ None cols(int) const { return {}; }
  __device__ __forceinline__ None ahead(int, int) const { return {}; }
  __device__ __forceinline__ void put(int m, int n, const f32x4& g, const f32x4& u, None, None) const {
    float h4[4], a4[4], b4[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float f, df;
      act_slope<!F32>(g[c], act, f, df);
      const bool in = n + c < N;
      a4[c] = in ? f : 0.0f;
      h4[c] = in ? f * u[c] : 0.0f;
      b4[c] = in ? u[c] * df : 0.0f;
    }
    const size_t o = static_cast<size_t>(m) * ld + n;
    store4<F32>(h, o, h4);
    const bool end = n + 4 >= N && (n & 4) == 0;
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    if (end) store4<F32>(h, o + 4, zero);
    if constexpr (!F32) {
      if (rests) {
        float r4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float r = bf16_bits_to_f32(f32_to_bf16_bits(h4[c]));
          r4[c] = isfinite(r) ? h4[c] - r : 0.0f;
        }
        store4<F32>(h, o + kRestRows * ld, r4);
        if (end) store4<F32>(h, o + kRestRows * ld + 4, zero);
      }
    }
    if constexpr (KEEP) {
      store4<true>(a, o, a4);
      store4<true>(b, o, b4);
    }
  }
};

// dg = dh b and du = dh a, side by side in rows of 2 ld.
template <bool F32>
struct SlopesOut {
  static constexpr int kAhead = 4;
  int bytes() const { return 8 + (F32 ? 8 : 4); }
  using Cols = None;
  struct Ahead {
    f32x4 a, b;
  };
  const float *a, *b;
  void* d;
  int64_t ld;
  int N;
  __device__ __forceinline__ None cols(int) const { return {}; }
  __device__ __forceinline__ Ahead ahead(int m, int n) const {
    const size_t o = static_cast<size_t>(m) * ld + n;
    return {load4<true>(a, o), load4<true>(b, o)};
  }
  __device__ __forceinline__ void put(int m, int n, const f32x4& s, const f32x4&, None, const Ahead& k) const {
    float g4[4], u4[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool in = n + c < N;
      g4[c] = in ? s[c] * k.b[c] : 0.0f;
      u4[c] = in ? s[c] * k.a[c] : 0.0f;
    }
    const size_t o = static_cast<size_t>(m) * 2 * ld + n;
    store4<F32>(d, o, g4);
    store4<F32>(d, o + ld, u4);
    // Both halves are contracted to their rows' ends.
    if (n + 4 >= N) {
      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
      for (int64_t k = n + 4; k < ld; k += 4) {
        store4<F32>(d, o - n + k, zero);
        store4<F32>(d, o - n + ld + k, zero);
      }
    }
  }
};

// The sums as they are; rows [0, half) of the product are y's, rows [half, 2 half) y2's,
// of either the first `live`.
template <bool F32>
struct RowsOut {
  static constexpr int kAhead = 4;
  int bytes() const { return F32 ? 4 : 2; }
  using Cols = None;
  using Ahead = None;
  void *y, *y2;
  int64_t ld;
  int N, half, live;
  __device__ __forceinline__ None cols(int) const { return {}; }
  __device__ __forceinline__ None ahead(int, int) const { return {}; }
  __device__ __forceinline__ void put(int m, int n, const f32x4& s, const f32x4&, None, None) const {
    const int r = m < half ? m : m - half;
    if (r >= live) return;
    const float v[4] = {s[0], s[1], s[2], s[3]};
    put4<F32>(m < half ? y : y2, static_cast<size_t>(r) * ld + n, v, N - n);
  }
};

// ---------------------------------------------------------------- zeros

// n bytes of zeros (a weight's gradient from no rows).
__global__ void __launch_bounds__(256) ffn_zero_kernel(uint8_t* p, size_t n) {
  for (size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 2; i < n; i += static_cast<size_t>(gridDim.x) * 512)
    *reinterpret_cast<uint16_t*>(p + i) = 0;
}

// ---------------------------------------------------------------- host

int check_ffn(const moe_ffn_config* c, int32_t rows) {
  if (!c) return MOE_ERR_NULL_PTR;
  if (c->dtype != MOE_DTYPE_F32 && c->dtype != MOE_DTYPE_BF16) return MOE_ERR_BAD_DTYPE;
  if (c->hidden_size <= 0 || c->intermediate_size <= 0 || rows < 0) return MOE_ERR_BAD_SHAPE;
  if (c->activation < MOE_ACT_NONE || c->activation > MOE_ACT_SILU) return MOE_ERR_BAD_SHAPE;
  // Grid and index arithmetic inside the kernels.
  if (c->hidden_size > MOE_LINEAR_MAX_FEATURES || c->intermediate_size > MOE_LINEAR_MAX_FEATURES / 4 ||
      rows > MOE_LINEAR_MAX_ROWS)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t type_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
// Length of the rows of h, a and b: whole stages of a contraction over them.
int64_t inner_ld(const moe_ffn_config& c) { return (static_cast<int64_t>(c.intermediate_size) + 63) / 64 * 64; }

// The kept tensors: h (of few rows with their rests), a, b.
bool with_rests(const moe_ffn_config& c, int64_t T) { return c.dtype == MOE_DTYPE_BF16 && T <= kRestRows; }
size_t h_bytes(const moe_ffn_config& c, int64_t T) {
  return align_up(static_cast<size_t>(std::max<int64_t>(T, 2 * kRestRows)) * inner_ld(c) * type_bytes(c.dtype), 256);
}
size_t slope_bytes(const moe_ffn_config& c, int64_t T) { return align_up(static_cast<size_t>(T) * inner_ld(c) * 4, 256); }
size_t kept_bytes(const moe_ffn_config& c, int64_t T) { return h_bytes(c, T) + 2 * slope_bytes(c, T); }

// Rows that do not lie in whole 16-byte pieces are laid out afresh, in one launch, for the
// products of more than 16 rows: loads of odd rows take in less than half as much.  A
// training step of 1001 x 1537 x 2049 takes 290 us with the rows as they lie, 151 to 172 with
// 2 x 11 to 12 for laying them out; forward and backward of 256 x 515 x 1023 27 + 45 and 22 + 39, of
// 64 x 129 x 257 17.9 + 40.3 and 16.2 + 36.4, of 17 x 65 x 129 13.7 + 31.7 and 14.4 + 27.8.  Room
// for x and dy is always there, room for the weights where their sizes are odd.
constexpr int64_t kPackFrom = int64_t{1} << 20;      // multiply-adds of a product, forward
int64_t eights(int64_t n) { return (n + 7) / 8 * 8; }
bool packs(const moe_ffn_config& c, int64_t T, bool backward) {
  return c.dtype == MOE_DTYPE_BF16 && T > kSkinnyRows && (backward || T * c.hidden_size * c.intermediate_size >= kPackFrom);
}
bool odd_sizes(const moe_ffn_config& c) { return c.hidden_size % 8 || c.intermediate_size % 8; }
// Rows of whole 128-byte lines, of which a stage takes one.
int64_t packed_ld(int64_t n) { return (n + 63) / 64 * 64; }
size_t packed_bytes(int64_t rows, int64_t n) { return align_up(static_cast<size_t>(rows) * packed_ld(n) * 2, 256); }

// The workspace: partial sums, then h (forward) or [dg du] (backward), then x, dy
// (backward), gate, up and down laid out afresh.
size_t ffn_parts(const moe_ffn_config& c, int64_t T) {
  const int64_t H = eights(c.hidden_size), Ip = inner_ld(c);
  const size_t n = std::max({part_bytes(true, T, Ip), part_bytes(false, T, Ip), part_bytes(false, T, H), part_bytes(false, 2 * Ip, H), part_bytes(false, H, Ip)});
  return align_up(n, 256);
}
size_t ffn_workspace(const moe_ffn_config& c, int64_t T, bool backward) {
  size_t n = ffn_parts(c, T) + (backward ? 2 : 1) * h_bytes(c, T);
  const int64_t H = eights(c.hidden_size), I = eights(c.intermediate_size);
  // Of any smaller number of rows too: the weights' room does not depend on it.
  if (c.dtype == MOE_DTYPE_BF16)
    n += (backward ? 2 : 1) * packed_bytes(T, H) + (odd_sizes(c) ? 2 * packed_bytes(I, H) + packed_bytes(H, I) : 0);
  return n;
}

bool misaligned(const void* p, size_t unit) { return reinterpret_cast<uintptr_t>(p) % unit != 0; }
constexpr int64_t kFar = int64_t{1} << 40;     // strides whose products with a row index stay in 64 bits

struct FfnArgs {
  const void *x, *dy, *wg, *wu, *wd;
  int64_t ldx, lddy, ldw, ldd;       // of x, dy, gate and up, down
  int H, I;                          // of the products: the sizes, or whole pieces of them
};

// The operands as they lie, or laid out afresh behind `room`.
int ffn_operands(const moe_ffn_config& c, int T, const void* x, int64_t ldx, const void* dy, int64_t lddy, const void* wg,
                 const void* wu, const void* wd, uint8_t* room, hipStream_t s, FfnArgs& f) {
  f = FfnArgs{x, dy, wg, wu, wd, ldx, lddy, c.hidden_size, c.intermediate_size, c.hidden_size, c.intermediate_size};
  if (!packs(c, T, dy != nullptr)) return MOE_OK;
  const bool odd = odd_sizes(c);
  const int H = c.hidden_size, I = c.intermediate_size, Hp = static_cast<int>(eights(H)), Ip = static_cast<int>(eights(I));
  const auto lies_odd = [](const void* p, int64_t ld) { return ld % 8 || reinterpret_cast<uintptr_t>(p) % 16; };
  PackArgs a{};
  const auto pack = [&](const void*& p, int64_t& ld, int rows, int cols, int to_rows, int to_cols) {
    a.item[a.n++] = PackItem{p, room, ld, packed_ld(to_cols), rows, cols, to_rows};
    p = room;
    ld = packed_ld(to_cols);
    room += packed_bytes(to_rows, to_cols);
  };
  if (odd || lies_odd(x, ldx)) pack(f.x, f.ldx, T, H, T, Hp);
  if (dy && (odd || lies_odd(dy, lddy))) pack(f.dy, f.lddy, T, H, T, Hp);
  if (odd) {
    pack(f.wg, f.ldw, I, H, Ip, Hp);
    f.ldw = H;
    pack(f.wu, f.ldw, I, H, Ip, Hp);
    pack(f.wd, f.ldd, H, I, Hp, Ip);
    f.H = Hp;
    f.I = Ip;
  }
  return a.n == 0 || pack_rows<uint16_t>(a, s) ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
}

template <bool F32>
int ffn_forward(const moe_ffn_config& c, int T, const FfnArgs& f, void* y, int64_t ldy, void* h, float* a, float* b,
                uint8_t* ws, hipStream_t s) {
  constexpr El E = F32 ? El::F32 : El::BF16;
  const int H = c.hidden_size, I = c.intermediate_size;
  const int64_t Ip = inner_ld(c);
  const Product g{{f.x, nullptr, f.ldx, 0, 0}, {f.wg, f.wu, f.ldw, 0, 0}, T, I, f.H};
  float* part = reinterpret_cast<float*>(ws);
  const bool rests = with_rests(c, T);
  const int st = a ? run_product<E, true, true, true>(g, GatedOut<F32, true>{h, a, b, Ip, I, c.activation, rests}, part, s)
                   : run_product<E, true, true, true>(g, GatedOut<F32, false>{h, a, b, Ip, I, c.activation, rests}, part, s);
  if (st) return st;
  const Product d{{h, nullptr, Ip, 0, 0}, {f.wd, nullptr, f.ldd, 0, 0}, T, H, f.I};
  const RowsOut<F32> out{y, nullptr, ldy, H, T, T};
  if constexpr (!F32) {
    const bool aligned = aligned16(d.a, E, true, T, f.I) && aligned16(d.b, E, true, H, f.I);
    if (rests) return launch_skinny<E, false>(d, out, aligned, part, s, WithRests{});
  }
  return run_product<E, true, true, false>(d, out, part, s);
}

template <bool F32>
int ffn_backward(const moe_ffn_config& c, int T, const FfnArgs& f, const void* h, const float* a, const float* b, void* dx,
                 int64_t lddx, void* dwg, void* dwu, void* dwd, void* d, uint8_t* ws, hipStream_t s) {
  constexpr El E = F32 ? El::F32 : El::BF16;
  const int H = c.hidden_size, I = c.intermediate_size, Ip = static_cast<int>(inner_ld(c));
  float* part = reinterpret_cast<float*>(ws);
  int st = MOE_OK;
  if (dwd) {
    const Product g{{f.dy, nullptr, f.lddy, 0, 0}, {h, nullptr, Ip, 0, 0}, f.H, f.I, T};
    st = run_product<E, false, false, false>(g, RowsOut<F32>{dwd, nullptr, I, I, f.H, H}, part, s);
  }
  if (st == MOE_OK && (dx || dwg)) {
    const Product g{{f.dy, nullptr, f.lddy, 0, 0}, {f.wd, nullptr, f.ldd, 0, 0}, T, f.I, f.H};
    st = run_product<E, true, false, false>(g, SlopesOut<F32>{a, b, d, Ip, I}, part, s);
  }
  if (st == MOE_OK && dwg) {
    const Product g{{d, nullptr, 2 * Ip, 0, 0}, {f.x, nullptr, f.ldx, 0, 0}, 2 * Ip, f.H, T};
    st = run_product<E, false, false, false>(g, RowsOut<F32>{dwg, dwu, H, H, Ip, I}, part, s);
  }
  if (st == MOE_OK && dx) {
    const Product g{{d, nullptr, 2 * Ip, 0, 0}, {f.wg, f.wu, f.ldw, Ip, I}, T, f.H, 2 * Ip};
    st = run_product<E, true, false, true>(g, RowsOut<F32>{dx, nullptr, lddx, H, T, T}, part, s);
  }
  return st;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_ffn_workspace_size(const moe_ffn_config* cfg, int32_t max_rows, int32_t backward, size_t* bytes) {
  const int st = check_ffn(cfg, max_rows);
  if (st) return st;
  if (!bytes) return MOE_ERR_NULL_PTR;
  *bytes = ffn_workspace(*cfg, max_rows, backward != 0);
  return MOE_OK;
}

int moe_ffn_kept_size(const moe_ffn_config* cfg, int32_t max_rows, size_t* bytes) {
  const int st = check_ffn(cfg, max_rows);
  if (st) return st;
  if (!bytes) return MOE_ERR_NULL_PTR;
  *bytes = std::max<size_t>(kept_bytes(*cfg, max_rows), 256);
  return MOE_OK;
}

int moe_ffn_forward(const moe_ffn_config* cfg, int32_t T, const void* x, int64_t ldx, const void* w_gate,
                    const void* w_up, const void* w_down, void* y, int64_t ldy, void* kept, size_t kept_size,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_ffn(cfg, T);
  if (st) return st;
  if (T == 0) return MOE_OK;
  if (!x || !w_gate || !w_up || !w_down || !y || !workspace) return MOE_ERR_NULL_PTR;
  if (ldx < cfg->hidden_size || ldy < cfg->hidden_size) return MOE_ERR_BAD_SHAPE;
  if (ldx > kFar || ldy > kFar) return MOE_ERR_UNSUPPORTED;
  if (workspace_bytes < ffn_workspace(*cfg, T, false)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (kept && kept_size < kept_bytes(*cfg, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const size_t e = type_bytes(cfg->dtype);
  if (misaligned(x, e) || misaligned(w_gate, e) || misaligned(w_up, e) || misaligned(w_down, e) || misaligned(y, e) ||
      misaligned(workspace, 16) || misaligned(kept, 16))
    return MOE_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* k = static_cast<uint8_t*>(kept);
  void* h = kept ? k : ws + ffn_parts(*cfg, T);
  float* a = kept ? reinterpret_cast<float*>(k + h_bytes(*cfg, T)) : nullptr;
  float* b = kept ? reinterpret_cast<float*>(k + h_bytes(*cfg, T) + slope_bytes(*cfg, T)) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  FfnArgs f;
  const int bad = ffn_operands(*cfg, T, x, ldx, nullptr, 0, w_gate, w_up, w_down, ws + ffn_parts(*cfg, T) + h_bytes(*cfg, T), s, f);
  if (bad) return bad;
  return cfg->dtype == MOE_DTYPE_F32 ? ffn_forward<true>(*cfg, T, f, y, ldy, h, a, b, ws, s)
                                     : ffn_forward<false>(*cfg, T, f, y, ldy, h, a, b, ws, s);
}

int moe_ffn_backward(const moe_ffn_config* cfg, int32_t T, const void* x, int64_t ldx, const void* w_gate,
                     const void* w_up, const void* w_down, const void* kept, size_t kept_size, const void* dy,
                     int64_t lddy, void* dx, int64_t lddx, void* dw_gate, void* dw_up, void* dw_down, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const int st = check_ffn(cfg, T);
  if (st) return st;
  if (!dw_gate != !dw_up) return MOE_ERR_NULL_PTR;
  const size_t e = type_bytes(cfg->dtype);
  if (misaligned(dx, e) || misaligned(dw_gate, e) || misaligned(dw_up, e) || misaligned(dw_down, e)) return MOE_ERR_UNSUPPORTED;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T == 0) {
    const size_t n = static_cast<size_t>(cfg->hidden_size) * cfg->intermediate_size * e;
    const unsigned grid = static_cast<unsigned>(std::min<size_t>(2048, (n + 511) / 512));
    for (void* w : {dw_gate, dw_up, dw_down})
      if (w) {
        ffn_zero_kernel<<<grid, 256, 0, s>>>(static_cast<uint8_t*>(w), n);
        if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
      }
    return MOE_OK;
  }
  if (!x || !w_gate || !w_up || !w_down || !kept || !dy || !workspace) return MOE_ERR_NULL_PTR;
  if (ldx < cfg->hidden_size || lddy < cfg->hidden_size || (dx && lddx < cfg->hidden_size)) return MOE_ERR_BAD_SHAPE;
  if (ldx > kFar || lddy > kFar || (dx && lddx > kFar)) return MOE_ERR_UNSUPPORTED;
  if (workspace_bytes < ffn_workspace(*cfg, T, true)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (kept_size < kept_bytes(*cfg, T)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (misaligned(x, e) || misaligned(w_gate, e) || misaligned(w_up, e) || misaligned(w_down, e) || misaligned(dy, e) ||
      misaligned(workspace, 16) || misaligned(kept, 16))
    return MOE_ERR_UNSUPPORTED;
  const uint8_t* k = static_cast<const uint8_t*>(kept);
  const float* a = reinterpret_cast<const float*>(k + h_bytes(*cfg, T));
  const float* b = reinterpret_cast<const float*>(k + h_bytes(*cfg, T) + slope_bytes(*cfg, T));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* d = ws + ffn_parts(*cfg, T);
  FfnArgs f;
  const int bad = ffn_operands(*cfg, T, x, ldx, dy, lddy, w_gate, w_up, w_down, d + 2 * h_bytes(*cfg, T), s, f);
  if (bad) return bad;
  return cfg->dtype == MOE_DTYPE_F32 ? ffn_backward<true>(*cfg, T, f, k, a, b, dx, lddx, dw_gate, dw_up, dw_down, d, ws, s)
                                     : ffn_backward<false>(*cfg, T, f, k, a, b, dx, lddx, dw_gate, dw_up, dw_down, d, ws, s);
}

}  // extern "C"
