// The whole layer for at most 16 tokens, in two kernels.
//
// With so few tokens the layer is the reading of its weights once from HBM: the
// router's, the touched experts' and the shared expert's.  What is lost on the way
// is lost between kernels, where the memory stands idle while one grid drains and
// the next fills, so the layer runs as two grids:
//
//   few_first_kernel   what does not depend on the routing: the router logits, split
//                      over the contraction, and the shared expert's gate/up half.
//                      It also clears the counters of the second kernel.
//   few_second_kernel  every workgroup works the routing out from the logits by
//                      itself (16 tokens: a few microseconds, no grid-wide step),
//                      then takes work items from a counter: first the gate/up
//                      items of the touched experts, then the down items, which
//                      contract over all touched experts and the shared expert at
//                      once, so that y leaves the kernel finished.
//
// All tokens are the 16 rows of one MFMA tile, whatever expert they go to; a row
// that an expert does not serve is zero there and its result is not used.  That
// spares the gather and the permutation, and costs nothing: the matrix cores idle.
//
// Waiting.  A down item needs every gate/up item's h.  Items are handed out by an
// atomic counter in order, gate/up items first, so when a workgroup holds a down
// item every gate/up item has been taken by a workgroup that is running, and
// gate/up items wait for nothing: the wait ends whatever part of the grid is
// resident, also when other kernels share the GPU.
//
// y is the same from run to run: every sum has a fixed order (the counters only say
// when something is complete).
//
// h leaves the gate/up half as two bf16 planes, h = hi + lo (16 significant bits;
// f32 layers keep one f32 plane): the second plane costs an L2 read and a second
// MFMA, both idle here, and takes the rounding of h out of y.
#include <algorithm>

#include "moe_mi355x.h"
#include "skinny.h"

namespace moe {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / kWave;
constexpr int kFewTokens = MOE_FEW_TOKENS;
static_assert(kFewTokens == kSkinnyRows, "one MFMA tile of tokens");
constexpr int kFewSlots = kFewTokens * kMaxTopK;
constexpr int kFewGrid = 512;              // two workgroups of eight waves on each of 256 CUs
constexpr int kFewRouterParts = 8;         // contraction parts of the router, at most

struct FewArgs {
  const void *x, *w_router, *w_gcol;
  const float* bias;
  const void *w_gate, *w_up, *w_down, *ws_gate, *ws_up, *ws_down;
  const void *s_gate, *s_up, *s_down, *ss_gate, *ss_up, *ss_down;
  int32_t* topk_ids;       // the outputs may be null, except one of y and y_act
  float* topk_w;
  float* shared_gate;
  int32_t* stats;
  float* y;
  void* y_act;
  int act_bf16;
  int* ctl;                // counters: next item, finished gate/up items
  float* z;                // [parts, 16, ldz] partial logits
  void *h, *h_lo;          // [T*K, I] routed then [T, S] shared
  int T, H, E, I, K, S, ncols, ldz, parts, norm, budget;
  float top_p;
  int rvec, hvec, ivec, svec;   // f32: rows of that length can be read in 16-byte pieces
};

// ---------------------------------------------------------------- pieces of both kernels

// Partial sums of the waves of a workgroup, one 16 x 16 tile each; a tile is added
// up in the order of the waves.
struct Red {
  f32x4 v[kFewWaves][kWave];
};

__device__ __forceinline__ f32x4 red_sum(const Red& r, int lane) {
  f32x4 s = r.v[0][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) {
    const f32x4 o = r.v[w][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += o[i];
  }
  return s;
}

template <int FMT>
struct GuBlk {
  WBlk<FMT> w;
  XBlk<FMT> x;
};

// This wave's eighth of x W^T over the contraction [b0, b1), in blocks, of one
// 16-row weight tile.
template <int FMT>
__device__ __forceinline__ f32x4 wave_tile(const WRow& row, const void* xrow, bool live, int b0, int b1, int kdim,
                                           bool vec, int wave, int g) {
  const int n = b1 - b0;
  const int lo = b0 + wave * n / kFewWaves, hi = b0 + (wave + 1) * n / kFewWaves;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  two_ahead<GuBlk<FMT>>(
      hi - lo,
      [&](int i, GuBlk<FMT>& k) {
        load_w<FMT>(k.w, row, lo + i, g, kdim, vec);
        load_x<FMT>(k.x, xrow, lo + i, g, kdim, vec, live);
      },
      [&](int, GuBlk<FMT>& k) { mma_block<FMT>(k.x, k.w, acc); });
  return acc;
}

template <int FMT>
__device__ __forceinline__ size_t row_bytes(int k) {
  return FMT == kDtypeF32 ? static_cast<size_t>(k) * 4
       : FMT == kDtypeBf16 ? static_cast<size_t>(k) * 2
       : FMT == kDtypeFp8 ? static_cast<size_t>(k) : static_cast<size_t>(k) / 2;
}
template <int FMT>
__device__ __forceinline__ size_t scale_bytes(int k) {
  return FMT == kDtypeFp8 ? static_cast<size_t>(k) / kGroup * 4
       : FMT == kDtypeMxfp4 ? static_cast<size_t>(k) / kMxBlock : 0;
}
template <int FMT>
__device__ __forceinline__ WRow weight_row(const void* w, const void* s, size_t row, int k) {
  return WRow{static_cast<const uint8_t*>(w) + row * row_bytes<FMT>(k),
              static_cast<const uint8_t*>(s) + row * scale_bytes<FMT>(k)};
}

// Columns [n0, n0 + 8) of a gate/up half: weight rows 0..7 of the tile are gate
// rows, 8..15 the up rows of the same columns (past the width: the last row again,
// not stored).
template <int FMT>
__device__ __forceinline__ WRow gate_up_row(const void* wg, const void* wu, const void* sg, const void* su,
                                            size_t first, int n0, int width, int H, int r) {
  const size_t row = first + min(n0 + (r & 7), width - 1);
  return r < 8 ? weight_row<FMT>(wg, sg, row, H) : weight_row<FMT>(wu, su, row, H);
}

// SwiGLU of a summed gate/up tile, written to h.  Lane l of a tile holds weight row
// l % 16 of tokens 4 (l / 16) + i; at(token) is the token's row of h, or -1.
template <int FMT, class At>
__device__ __forceinline__ void store_h(const FewArgs& a, const f32x4& s, size_t base, int n0, int width, int lane,
                                        At at) {
  const int r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float up = __shfl_xor(s[i], 8, kWave);
    const int row = at(4 * g + i);
    if (r < 8 && n0 + r < width && row >= 0) {
      const float h = s[i] / (1.0f + expf(-s[i])) * up;
      const size_t o = base + static_cast<size_t>(row) * width + n0 + r;
      if constexpr (FMT == kDtypeF32) {
        static_cast<float*>(a.h)[o] = h;
      } else {
        const uint16_t hi = f32_to_bf16_bits(h);
        const float back = bf16_bits_to_f32(hi);
        static_cast<uint16_t*>(a.h)[o] = hi;
        // An infinite hi has no remainder (inf - inf would turn it into NaN).
        static_cast<uint16_t*>(a.h_lo)[o] = fabsf(back) < INFINITY ? f32_to_bf16_bits(h - back) : 0;
      }
    }
  }
}

// ---------------------------------------------------------------- first kernel

template <int FMT>
__global__ void __launch_bounds__(kFewThreads) few_first_kernel(FewArgs a) {
  constexpr int AFMT = FMT == kDtypeF32 ? kDtypeF32 : kDtypeBf16;   // the router's type
  __shared__ Red red;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  if (blockIdx.x == 0 && tid < 2) a.ctl[tid] = 0;

  const size_t xrow_bytes = static_cast<size_t>(a.H) * (AFMT == kDtypeF32 ? 4 : 2);
  const void* xrow = static_cast<const uint8_t*>(a.x) + static_cast<size_t>(min(r, a.T - 1)) * xrow_bytes;
  const bool live = r < a.T;
  const int router = static_cast<int>(ceil_div(a.ncols, 16)) * a.parts;
  int item = blockIdx.x;
  if (item < router) {
    const int part = item % a.parts, c0 = item / a.parts * 16;
    const int nb = static_cast<int>(ceil_div(a.H, SkinnyFmt<AFMT>::kBlk));
    const int c = min(c0 + r, a.ncols - 1);
    const WRow row = c < a.E ? weight_row<AFMT>(a.w_router, nullptr, c, a.H) : WRow{static_cast<const uint8_t*>(a.w_gcol), nullptr};
    red.v[wave][lane] = wave_tile<AFMT>(row, xrow, live, part * nb / a.parts, (part + 1) * nb / a.parts, a.H,
                                        a.rvec, wave, g);
    __syncthreads();
    if (wave == 0 && c0 + r < a.ncols) {
      const f32x4 s = red_sum(red, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a.z[(static_cast<size_t>(part) * kFewTokens + 4 * g + i) * a.ldz + c0 + r] = s[i];
    }
    return;
  }
  const int n0 = (item - router) * 8;
  const WRow row = gate_up_row<FMT>(a.ws_gate, a.ws_up, a.ss_gate, a.ss_up, 0, n0, a.S, a.H, r);
  red.v[wave][lane] = wave_tile<FMT>(row, xrow, live, 0, static_cast<int>(ceil_div(a.H, SkinnyFmt<FMT>::kBlk)), a.H,
                                     a.hvec, wave, g);
  __syncthreads();
  if (wave == 0) {
    const f32x4 s = red_sum(red, lane);
    store_h<FMT>(a, s, static_cast<size_t>(a.T) * a.K * a.I, n0, a.S, lane,
                 [&](int t) { return t < a.T ? t : -1; });
  }
}

// ---------------------------------------------------------------- routing

// The order of floats as unsigned integers; 0 is below every float.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);     // -0 and +0 are equal
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      static_cast<int>(v), static_cast<int>(v), CTRL, 0xf, 0xf, false));
  return max(v, o);
}
// Maximum over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max<0x111>(v);      // row_shr 1, 2, 4, 8: lane 15 of each row of 16
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);      // row_bcast 15, 31: lane 63
  v = dpp_max<0x143>(v);
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

constexpr double kFewFixed = 8589934592.0;   // 2^33: budget aggregates in fixed point, as in moe_route

// What every workgroup knows of the call's routing.
struct Routing {
  int ids[kFewSlots];              // [T, K]
  float w[kFewSlots];
  float sg[kFewTokens];            // sigmoid of the shared gate
  int n;                           // touched experts
  int seg_expert[kFewSlots];
  int16_t seg_slot[kFewSlots + 1][kFewTokens];   // row of h of (segment, token), -1: not served
  float seg_w[kFewSlots + 1][kFewTokens];        // its weight, 0 if not served
};
struct RouteScratch {
  unsigned long long agg[kMaxExperts];
  int seg_of[kMaxExperts];
  int nu, dropped, empty;
  int list[kFewSlots];
};

// Same selection, trim and budget as moe_route.
__device__ void route_tokens(const FewArgs& a, Routing& R, RouteScratch& C, bool report) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t plane = static_cast<size_t>(kFewTokens) * a.ldz;
  constexpr int NJ = kMaxExperts / kWave;
  for (int t = wave; t < a.T; t += kFewWaves) {
    const float* zr = a.z + static_cast<size_t>(t) * a.ldz;
    auto logit = [&](int c) {
      float s = zr[c];
      for (int p = 1; p < a.parts; ++p) s += zr[p * plane + c];
      return s;
    };
    const float gate_logit = (a.S > 0 && lane == 0) ? logit(a.E) : 0.f;
    uint32_t key[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + kWave * j;
      key[j] = 0;
      if (e < a.E) {
        float v = logit(e);
        if (a.bias) v += a.bias[static_cast<size_t>(t) * a.E + e];
        key[j] = order_key(v == v ? v : -INFINITY);
      }
    }
    // Softmax denominator over all experts (only without renormalisation).
    float denom_all = 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) top = max(top, key[j]);
    const float zmax = key_value(wave_max_u32(top));
    if (!a.norm) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (lane + kWave * j < a.E) denom_all += expf(key_value(key[j]) - zmax);
      denom_all = wave_sum(denom_all);
    }
    int my_id = -1;
    float my_z = 0.f;
    for (int k = 0; k < a.K; ++k) {
      uint32_t best = 0;
#pragma unroll
      for (int j = 0; j < NJ; ++j) best = max(best, key[j]);
      const uint32_t m = wave_max_u32(best);
      // The lowest id that holds it: ids grow with j, then with the lane.
      int id = 0x7fffffff;
#pragma unroll
      for (int j = NJ - 1; j >= 0; --j) {
        const unsigned long long has = __ballot(key[j] == m);
        if (has) id = kWave * j + __builtin_ctzll(has);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (lane + kWave * j == id) key[j] = 0;
      if (lane == k) { my_id = id; my_z = key_value(m); }
    }
    const float p = lane < a.K ? expf(my_z - zmax) : 0.f;
    bool kept = lane < a.K;
    if (a.top_p > 0.f) {
      float before = 0.f, all = 0.f;
      for (int k = 0; k < a.K; ++k) {
        const float pk = __shfl(p, k, kWave);
        if (k < lane) before += pk;
        all += pk;
      }
      kept = kept && (lane == 0 || before < a.top_p * all);
    }
    const float pk = kept ? p : 0.f;
    const float denom = a.norm ? wave_sum(pk) : denom_all;
    if (lane < a.K) {
      R.ids[t * a.K + lane] = kept ? my_id : -1;
      R.w[t * a.K + lane] = pk / denom;
    }
    if (lane == 0) R.sg[t] = a.S > 0 ? 1.0f / (1.0f + expf(-gate_logit)) : 0.f;
  }
  const int slots = a.T * a.K;
  for (int e = tid; e < kMaxExperts; e += kFewThreads) { C.agg[e] = 0ull; C.seg_of[e] = 0; }
  if (tid == 0) { C.nu = 0; C.dropped = 0; C.empty = 0; }
  __syncthreads();

  // Expert budget.  seg_of marks presence here.
  if (a.budget > 0 || (report && a.stats)) {
    for (int i = tid; i < slots; i += kFewThreads) {
      const int e = R.ids[i];
      if (e >= 0) {
        const float w = R.w[i];
        if (w == w) atomicAdd(&C.agg[e], static_cast<unsigned long long>(llrint(static_cast<double>(w) * kFewFixed)));
        if (atomicExch(&C.seg_of[e], 1) == 0) C.list[atomicAdd(&C.nu, 1)] = e;
      }
    }
    __syncthreads();
    const int nu = C.nu;
    const bool active = a.budget > 0 && nu > a.budget;
    if (active) {
      int e = -1, rank = 0;
      if (tid < nu) {
        e = C.list[tid];
        const unsigned long long v = C.agg[e];
        for (int o = 0; o < nu; ++o) {
          const int f = C.list[o];
          const unsigned long long u = C.agg[f];
          rank += (u > v || (u == v && f < e)) ? 1 : 0;
        }
      }
      __syncthreads();
      if (e >= 0) C.seg_of[e] = rank < a.budget ? 1 : 0;
      __syncthreads();
      if (tid < a.T) {
        int* ir = R.ids + tid * a.K;
        float* wr = R.w + tid * a.K;
        int nk = 0, nd = 0;
        float sum = 0.f;
        for (int k = 0; k < a.K; ++k) {
          if (ir[k] < 0) continue;
          if (C.seg_of[ir[k]]) { sum += wr[k]; ++nk; } else { ++nd; }
        }
        if (nd) {
          int j = 0;
          for (int k = 0; k < a.K; ++k) {
            const int e2 = ir[k];
            if (e2 >= 0 && C.seg_of[e2]) {
              const float v = wr[k];
              ir[j] = e2;
              wr[j] = a.norm ? v / sum : v;
              ++j;
            }
          }
          for (; j < a.K; ++j) { ir[j] = -1; wr[j] = 0.f; }
          atomicAdd(&C.dropped, nd);
        }
        if (nk == 0) atomicAdd(&C.empty, 1);
      }
      __syncthreads();
    }
    if (report && a.stats && tid == 0) {
      a.stats[0] = nu;
      a.stats[1] = active ? a.budget : nu;
      a.stats[2] = C.dropped;
      a.stats[3] = C.empty;
    }
    __syncthreads();
  }

  // Segments: the touched experts in ascending order.  A slot of weight 0 is not run.
  for (int e = tid; e < kMaxExperts; e += kFewThreads) C.seg_of[e] = 0;
  for (int i = tid; i < (kFewSlots + 1) * kFewTokens; i += kFewThreads) {
    (&R.seg_slot[0][0])[i] = -1;
    (&R.seg_w[0][0])[i] = 0.f;
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kFewThreads)
    if (R.ids[i] >= 0 && R.w[i] != 0.f) C.seg_of[R.ids[i]] = 1;
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int base = 0; base < a.E; base += kWave) {
      const int e = base + lane;
      const bool has = e < a.E && C.seg_of[e] != 0;
      const unsigned long long m = __ballot(has);
      if (has) {
        const int s = n + __popcll(m & ((1ull << lane) - 1));
        R.seg_expert[s] = e;
        C.seg_of[e] = s;
      }
      n += __popcll(m);
    }
    if (lane == 0) R.n = n;
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kFewThreads)
    if (R.ids[i] >= 0 && R.w[i] != 0.f) {
      const int s = C.seg_of[R.ids[i]], t = i / a.K;
      R.seg_slot[s][t] = static_cast<int16_t>(i);
      R.seg_w[s][t] = R.w[i];
    }
  // The shared expert is the segment after them: every token, weighted by its gate.
  if (a.S > 0 && tid < a.T) {
    R.seg_slot[R.n][tid] = static_cast<int16_t>(tid);
    R.seg_w[R.n][tid] = R.sg[tid];
  }
  if (report) {
    for (int i = tid; i < slots; i += kFewThreads) {
      if (a.topk_ids) a.topk_ids[i] = R.ids[i];
      if (a.topk_w) a.topk_w[i] = R.w[i];
    }
    if (a.shared_gate && a.S > 0 && tid < a.T) a.shared_gate[tid] = R.sg[tid];
  }
  __syncthreads();
}

// ---------------------------------------------------------------- second kernel

template <int FMT>
struct DownBlk {
  WBlk<FMT> w;
  XBlk<FMT> hi, lo;
};

template <int FMT>
__global__ void __launch_bounds__(kFewThreads, 4) few_second_kernel(FewArgs a) {
  using F = SkinnyFmt<FMT>;
  __shared__ Red red;
  __shared__ Routing R;
  __shared__ RouteScratch C;
  __shared__ int s_item;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  route_tokens(a, R, C, blockIdx.x == 0);

  const int n = R.n;
  const int hb = static_cast<int>(ceil_div(a.H, F::kBlk)), ib = static_cast<int>(ceil_div(a.I, F::kBlk)),
            sb = static_cast<int>(ceil_div(a.S, F::kBlk));
  const int gu_tiles = static_cast<int>(ceil_div(a.I, 8));
  const int gu_items = n * gu_tiles;
  const int total = gu_items + static_cast<int>(ceil_div(a.H, 16));
  const size_t h_shared = static_cast<size_t>(a.T) * a.K * a.I;
  bool ready = false;

  for (;;) {
    __syncthreads();                 // the previous item's red and s_item have been read
    if (tid == 0) s_item = __hip_atomic_fetch_add(&a.ctl[0], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const int item = __builtin_amdgcn_readfirstlane(s_item);
    if (item >= total) break;
    if (item < gu_items) {
      const int seg = item / gu_tiles, n0 = item % gu_tiles * 8;
      const int e = __builtin_amdgcn_readfirstlane(R.seg_expert[seg]);
      const WRow row = gate_up_row<FMT>(a.w_gate, a.w_up, a.s_gate, a.s_up, static_cast<size_t>(e) * a.I, n0, a.I,
                                        a.H, r);
      const void* xrow = static_cast<const uint8_t*>(a.x) + static_cast<size_t>(min(r, a.T - 1)) * a.H * (F::kF32 ? 4 : 2);
      red.v[wave][lane] = wave_tile<FMT>(row, xrow, R.seg_slot[seg][r] >= 0, 0, hb, a.H, a.hvec, wave, g);
      __syncthreads();
      if (wave == 0) {
        const f32x4 s = red_sum(red, lane);
        store_h<FMT>(a, s, 0, n0, a.I, lane, [&](int t) { return static_cast<int>(R.seg_slot[seg][t]); });
        // One wave wrote the item's h, so its release covers all of it.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        if (lane == 0) __hip_atomic_fetch_add(&a.ctl[1], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      continue;
    }
    if (!ready) {                    // uniform across the workgroup
      if (tid == 0)
        while (__hip_atomic_load(&a.ctl[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < gu_items)
          __builtin_amdgcn_s_sleep(1);
      __syncthreads();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      ready = true;
    }
    const int n0 = (item - gu_items) * 16;
    const int orow = min(n0 + r, a.H - 1);
    const int nblk = n * ib + (a.S > 0 ? sb : 0);
    const int lo = static_cast<int>(static_cast<int64_t>(wave) * nblk / kFewWaves);
    const int hi = static_cast<int>(static_cast<int64_t>(wave + 1) * nblk / kFewWaves);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    auto seg_of = [&](int b) { return min(b / ib, n); };
    two_ahead<DownBlk<FMT>>(
        hi - lo,
        [&](int i, DownBlk<FMT>& k) {
          const int b = lo + i, seg = seg_of(b), kb = b - seg * ib;
          const bool shared = seg == n;
          const int width = shared ? a.S : a.I;
          const size_t wrow = shared ? orow : static_cast<size_t>(R.seg_expert[seg]) * a.H + orow;
          const WRow row = weight_row<FMT>(shared ? a.ws_down : a.w_down, shared ? a.ss_down : a.s_down, wrow, width);
          const bool vec = shared ? a.svec : a.ivec;
          load_w<FMT>(k.w, row, kb, g, width, vec);
          const int slot = R.seg_slot[seg][r];
          const size_t ho = (shared ? h_shared : 0) + static_cast<size_t>(max(slot, 0)) * width;
          if constexpr (F::kF32) {
            load_x<FMT>(k.hi, static_cast<const float*>(a.h) + ho, kb, g, width, vec, slot >= 0);
          } else {
            load_x<FMT>(k.hi, static_cast<const uint16_t*>(a.h) + ho, kb, g, width, vec, slot >= 0);
            load_x<FMT>(k.lo, static_cast<const uint16_t*>(a.h_lo) + ho, kb, g, width, vec, slot >= 0);
          }
        },
        [&](int i, DownBlk<FMT>& k) {
          const int seg = seg_of(lo + i);
          f32x4 t = mma_raw<FMT>(k.hi, k.w, f32x4{0.f, 0.f, 0.f, 0.f});
          if constexpr (!F::kF32) t = mma_raw<FMT>(k.lo, k.w, t);
          const float4 w = *reinterpret_cast<const float4*>(&R.seg_w[seg][4 * g]);
          const float ws[4] = {w.x, w.y, w.z, w.w};
          // A token that the expert does not serve takes nothing, not 0 * inf either.
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v = FMT == kDtypeFp8 ? t[q] * k.w.s : t[q];
            acc[q] = ws[q] != 0.f ? fmaf(ws[q], v, acc[q]) : acc[q];
          }
        });
    red.v[wave][lane] = acc;
    __syncthreads();
    if (wave == 0 && n0 + r < a.H) {
      const f32x4 s = red_sum(red, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * g + i;
        if (t < a.T) {
          const size_t o = static_cast<size_t>(t) * a.H + n0 + r;
          if (a.y) a.y[o] = s[i];
          if (a.y_act) {
            if (a.act_bf16) static_cast<uint16_t*>(a.y_act)[o] = f32_to_bf16_bits(s[i]);
            else static_cast<float*>(a.y_act)[o] = s[i];
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- host

struct FewLayout {
  size_t ctl, z, h, h_lo, total;
  int ldz, parts;
};

FewLayout few_layout(const moe_config& c, int64_t T) {
  FewLayout L{};
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t o = off;
    off = align_up(off + n, 256);
    return o;
  };
  const bool f32 = c.weight_dtype == MOE_DTYPE_F32;
  L.ldz = static_cast<int>(align_up(c.n_routed_experts + 1, 16));
  // At least one block of contraction for each wave of a part.
  const int blocks = static_cast<int>(ceil_div(c.hidden_size, f32 ? 32 : 128));
  L.parts = std::max(1, std::min(kFewRouterParts, blocks / kFewWaves));
  L.ctl = take(2 * sizeof(int));
  L.z = take(static_cast<size_t>(L.parts) * kFewTokens * L.ldz * sizeof(float));
  const size_t elems = static_cast<size_t>(T) * c.num_experts_per_tok * c.moe_intermediate_size +
                       static_cast<size_t>(T) * c.shared_expert_intermediate_size;
  L.h = take(elems * (f32 ? 4 : 2));
  L.h_lo = take(f32 ? 0 : elems * 2);
  L.total = off;
  return L;
}

bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <int FMT>
int few_launch(const FewArgs& a, hipStream_t s) {
  const int first = static_cast<int>(ceil_div(a.ncols, 16)) * a.parts + static_cast<int>(ceil_div(a.S, 8));
  few_first_kernel<FMT><<<first, kFewThreads, 0, s>>>(a);
  if (hipGetLastError() != hipSuccess) return MOE_ERR_LAUNCH_FAILED;
  few_second_kernel<FMT><<<kFewGrid, kFewThreads, 0, s>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH_FAILED;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_layer_few_workspace_size(const moe_config* cfg, int32_t max_tokens, size_t* bytes) {
  size_t n = 0;
  const int st = moe_workspace_size(cfg, max_tokens, bytes ? &n : nullptr);   // the layer's checks
  if (st) return st;
  if (max_tokens > kFewTokens) return MOE_ERR_UNSUPPORTED;
  *bytes = few_layout(*cfg, max_tokens).total;
  return MOE_OK;
}

int moe_layer_few(const moe_config* cfg, int32_t T, const void* x, const void* w_router,
                  const void* w_shared_gate, const float* logit_bias, const moe_expert_weights* w,
                  int32_t* topk_ids, float* topk_weights, float* shared_gate, int32_t* route_stats, float* y,
                  void* y_act, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const int st = moe_layer_few_workspace_size(cfg, T, &need);
  if (st) return st;
  if (T == 0) return MOE_OK;
  const bool shared = cfg->shared_expert_intermediate_size > 0;
  const bool f32 = cfg->weight_dtype == MOE_DTYPE_F32;
  const bool quant = cfg->weight_dtype == MOE_DTYPE_FP8_E4M3_G128 || cfg->weight_dtype == MOE_DTYPE_MXFP4;
  if (!x || !w_router || !w || (!y && !y_act) || !workspace) return MOE_ERR_NULL_PTR;
  if (!w->w_gate || !w->w_up || !w->w_down) return MOE_ERR_NULL_PTR;
  if (quant && (!w->s_gate || !w->s_up || !w->s_down)) return MOE_ERR_NULL_PTR;
  if (shared && (!w_shared_gate || !w->ws_gate || !w->ws_up || !w->ws_down)) return MOE_ERR_NULL_PTR;
  if (shared && quant && (!w->ss_gate || !w->ss_up || !w->ss_down)) return MOE_ERR_NULL_PTR;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;

  // Operands are read in 16-byte pieces; f32 layers fall back to single elements.
  const uintptr_t unit = f32 ? 4 : 16;
  const uintptr_t scale = cfg->weight_dtype == MOE_DTYPE_FP8_E4M3_G128 ? 4 : 1;
  const void* rows[] = {x, w_router, w->w_gate, w->w_up, w->w_down};
  const void* srows[] = {w_shared_gate, w->ws_gate, w->ws_up, w->ws_down};
  const void* scales[] = {w->s_gate, w->s_up, w->s_down};
  const void* sscales[] = {w->ss_gate, w->ss_up, w->ss_down};
  bool bad = misaligned(workspace, 16) || misaligned(y, 4) || misaligned(y_act, f32 ? 4 : 2) ||
             misaligned(logit_bias, 4) || misaligned(topk_ids, 4) || misaligned(topk_weights, 4) ||
             misaligned(route_stats, 4);
  bool wide = true;          // f32: every operand 16-byte aligned
  for (const void* p : rows) { bad |= misaligned(p, unit); wide &= !misaligned(p, 16); }
  if (quant) for (const void* p : scales) bad |= misaligned(p, scale);
  if (shared) {
    for (const void* p : srows) { bad |= misaligned(p, unit); wide &= !misaligned(p, 16); }
    if (quant) for (const void* p : sscales) bad |= misaligned(p, scale);
    bad |= misaligned(shared_gate, 4);
  }
  if (bad) return MOE_ERR_UNSUPPORTED;

  const FewLayout L = few_layout(*cfg, T);
  char* ws = static_cast<char*>(workspace);
  FewArgs a{};
  a.x = x;
  a.w_router = w_router;
  a.w_gcol = w_shared_gate;
  a.bias = logit_bias;
  a.w_gate = w->w_gate; a.w_up = w->w_up; a.w_down = w->w_down;
  a.ws_gate = w->ws_gate; a.ws_up = w->ws_up; a.ws_down = w->ws_down;
  a.s_gate = w->s_gate; a.s_up = w->s_up; a.s_down = w->s_down;
  a.ss_gate = w->ss_gate; a.ss_up = w->ss_up; a.ss_down = w->ss_down;
  a.topk_ids = topk_ids;
  a.topk_w = topk_weights;
  a.shared_gate = shared_gate;
  a.stats = route_stats;
  a.y = y;
  a.y_act = y_act;
  a.act_bf16 = f32 ? 0 : 1;
  a.ctl = reinterpret_cast<int*>(ws + L.ctl);
  a.z = reinterpret_cast<float*>(ws + L.z);
  a.h = ws + L.h;
  a.h_lo = ws + L.h_lo;
  a.T = T;
  a.H = cfg->hidden_size;
  a.E = cfg->n_routed_experts;
  a.I = cfg->moe_intermediate_size;
  a.K = cfg->num_experts_per_tok;
  a.S = cfg->shared_expert_intermediate_size;
  a.ncols = a.E + (shared ? 1 : 0);
  a.ldz = L.ldz;
  a.parts = L.parts;
  a.norm = cfg->norm_topk_prob;
  a.budget = cfg->expert_budget;
  a.top_p = (cfg->top_p > 0.f && cfg->top_p < 1.f) ? cfg->top_p : 0.f;
  a.rvec = a.hvec = wide && a.H % 4 == 0;
  // h rows: the workspace is aligned, the shared rows start at T*K*I.
  a.ivec = wide && a.I % 4 == 0;
  a.svec = wide && a.S % 4 == 0 && (static_cast<int64_t>(T) * a.K * a.I) % 4 == 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (cfg->weight_dtype) {
    case MOE_DTYPE_F32: return few_launch<kDtypeF32>(a, s);
    case MOE_DTYPE_BF16: return few_launch<kDtypeBf16>(a, s);
    case MOE_DTYPE_FP8_E4M3_G128: return few_launch<kDtypeFp8>(a, s);
    default: return few_launch<kDtypeMxfp4>(a, s);
  }
}

}  // extern "C"
