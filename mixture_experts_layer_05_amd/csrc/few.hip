// The whole layer for at most 16 tokens, in two kernels.
//
// With so few tokens the layer is the reading of its weights once from HBM: the
// router's, the touched experts' and the shared expert's.  What is lost on the way
// is lost between kernels, where the memory stands idle while one grid drains and
// the next fills, so the layer runs as two grids:
//
//   few_first_kernel   the router logits, split over the contraction; it also clears
//                      the counters of the second kernel.
//   few_second_kernel  a few workgroups work the routing out from the logits and
//                      publish it; meanwhile the others run the shared expert's
//                      gate/up tiles, which do not depend on it.  Then the touched
//                      experts' gate/up tiles, and the down half, which contracts over
//                      all touched experts and the shared expert at once, so that y
//                      leaves the kernel finished.
//
// All tokens are the 16 rows of one MFMA tile, whatever expert they go to; a row
// that an expert does not serve is zero there and its result is not used.  That
// spares the gather and the permutation, and costs nothing: the matrix cores idle.
//
// Waiting.  The down half needs every gate/up tile.  The tiles are handed out from
// eight queues (one for each XCD; a workgroup whose own is empty takes from the
// others), so a tile that has been taken is held by a workgroup that is running, and
// that finishes it without waiting for anything.  A workgroup waits only when it has
// seen all queues empty: the wait ends, whatever part of the grid is resident, also
// when other kernels hold part of the GPU.  The wait for the published routing is
// bounded: a workgroup that does not find it in time works it out by itself.
//
// y is the same from run to run: every sum has a fixed order (queues and
// counters say who works and when something is complete, not in which order it is
// added).
//
// h leaves the gate/up half as three bf16 planes whose sum is its float32 value (f32
// layers keep one f32 plane).  With one plane its rounding would be the largest
// error in y by far; the others cost L2 reads and MFMAs that are idle here.
//
// What bounds it, measured (wall time of a call; a large copy moves 5.0 TB/s here):
//   256 experts, top-8, I 2048, H 7168, fp8, 16 tokens on 64 experts   2911 MB  553 to 568 us  5.2 TB/s
//   512 experts, top-10, I 512, S 2048, H 5120, bf16, 7 tokens         1108 MB  241 us  4.6 TB/s
//   the same in MXFP4, 16 tokens, top-p 0.9                             545 MB  161 to 168 us  3.3 TB/s
//   16 experts, top-2, I 1024, S 2048, H 5120, bf16, 7 tokens           260 MB   77 to 85 us  3.1 to 3.4 TB/s
//   the same, 1 token                                                   126 MB   50 us  2.5 TB/s
// The large calls are bound by the memory.  In the smallest the memory stands idle
// between the steps: with 1 token the router takes 6 us (on 4 workgroups, while the
// shared expert's weights wait), the routing 4, the gate/up half 20, the wait for the
// last h and the down weights 8 (which arrive meanwhile), h's loads 6, the parts' sum 2.
// In MXFP4 each decoded operand of the down half meets three planes of h: without the
// second and third the call above takes 150 of 168 us, the fp8 one 535 of 568, the
// bf16 one 232 of 241.  The rest above the memory's time is decoding, and pieces of 41 KB.
// Reading h past the caches instead of invalidating
// them saved 1 us of that with one token and cost up to 15 % with sixteen; a ring of
// loads in place of batches changed nothing, nor did longer batches in the down half.
#include <algorithm>
#include <cstddef>

#include "moe_mi355x.h"
#include "skinny.h"

namespace moe {
namespace {

// Two workgroups of four waves on each of 256 CUs, 256 registers per lane: while one
// workgroup adds a tile up the other one's loads keep the CU's memory path busy.
constexpr int kFewThreads = 256;
constexpr int kFewWaves = kFewThreads / kWave;
constexpr int kFewGrid = 512;
constexpr int kFewTokens = MOE_FEW_TOKENS;
static_assert(kFewTokens * kMaxTopK <= kFewThreads, "a thread for each slot");
static_assert(kFewTokens == kSkinnyRows, "one MFMA tile of tokens");
constexpr int kFewSlots = kFewTokens * kMaxTopK;
constexpr int kFewRouterParts = 4;         // contraction parts of the router, at most
constexpr int kQueues = 8;

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
  int* ctl;                // counters of the second kernel, see Ctl
  float* z;                // [parts, 16, ldz] partial logits
  void* h[3];              // planes of [T*K, I] routed then [T, S] shared rows
  int* routed;             // published routing: ids and weights [T, K], shared gates [T]
  float* part;             // [2 * kMaxRanges, sets, 256] partial down tiles
  int T, H, E, I, K, S, ldz, parts, norm, budget;
  float top_p;
  int hvec, ivec, svec;   // f32: rows of that length can be read in 16-byte pieces
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

// Blocks of weights that a wave loads at a time, within its 256 registers.  Where an
// activation block is large next to a weight block, several tiles run side by side on
// one: kWide in the gate/up half when there are enough tiles (kWideTiles for each
// workgroup), kSets in the down half, whose weights meet three planes of h.  With one
// tile at a time the activations' loads took a fifth to a third of the gate/up time of
// the quantised types.
template <int FMT>
struct FewBatch {
  static constexpr int kWide = FMT == kDtypeMxfp4 ? 4 : FMT == kDtypeF32 ? 1 : 2;
  static constexpr int kGateUp = FMT == kDtypeMxfp4 ? 4 : FMT == kDtypeFp8 ? 6 : 10;
  static constexpr int kGateUpWide = FMT == kDtypeMxfp4 ? 2 : FMT == kDtypeFp8 ? 4 : 5;
  static constexpr int kDown = FMT == kDtypeMxfp4 || FMT == kDtypeFp8 ? 1 : 4;
  static constexpr int kDownScales = FMT == kDtypeMxfp4 ? 2 : 4;   // blocks whose scales are loaded together
  static constexpr int kSets = FMT == kDtypeF32 ? 1 : FMT == kDtypeBf16 ? 2 : 4;
};
// 512 experts, top-10, I 512, H 5120, 9 tokens: 143 us with 16 tiles for each workgroup,
// 129 with 4 (mxfp4), 202 and 191 (fp8); with 2 the items became too few for 16 experts,
// top-2, I 1024, 16 tokens: 139 -> 144 us (bf16), 82 -> 86 (mxfp4).
constexpr int kWideTiles = 4;
constexpr int kMaxSets = 4;

// NS gate/up tiles side by side on one block of x.
template <int FMT, int NS>
struct GuBlk {
  WBlk<FMT> w[NS];
  XBlk<FMT> x[1];
};

// This wave's quarter of x W^T over the contraction [b0, b1), in blocks, of NS 16-row
// weight tiles.  first() is called when the loads of the first batch are on their way.
template <int FMT, int NS, class First>
__device__ __forceinline__ void wave_tiles(const Matrices& m, const WRow (&row)[NS], const void* x, uint32_t xoff,
                                           bool live, int b0, int b1, int kdim, bool vec, int wave, int lane,
                                           f32x4 (&acc)[NS], First first) {
  constexpr int D = NS == 1 ? FewBatch<FMT>::kGateUp : FewBatch<FMT>::kGateUpWide;
  const int n = b1 - b0;
  const int lo = b0 + wave * n / kFewWaves, hi = b0 + (wave + 1) * n / kFewWaves;
#pragma unroll
  for (int j = 0; j < NS; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (!Scales<FMT, 1>::kAny) {
    int at = lo;
    batches<D, GuBlk<FMT, NS>>(
        hi - lo,
        [&](GuBlk<FMT, NS>& k) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < NS; ++j) load_w<FMT>(k.w[j], m, row[j], at, lane, kdim, vec);
          load_x<FMT>(k.x[0], x, xoff, at, lane, kdim, vec, live);
          ++at;
        },
        [&](GuBlk<FMT, NS>& k) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < NS; ++j) acc[j] = mma_planes<FMT, 1>(k.x, k.w[j], lane, acc[j]);
        },
        first);
  } else {
    const int blocks = kdim / SkinnyFmt<FMT>::kBlk;      // of a row
    for (int c = lo; c < hi; c += D) {
      GuBlk<FMT, NS> k[D];
      Scales<FMT, D> sc[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) sc[j].load(row[j].s + blk_scale_bytes<FMT>() * c, blocks - c);
#pragma unroll
      for (int s = 0; s < D; ++s)
        if (c + s < hi) {
#pragma unroll
          for (int j = 0; j < NS; ++j) load_w<FMT>(k[s].w[j], m, row[j], c + s, lane, kdim, vec);
          load_x<FMT>(k[s].x[0], x, xoff, c + s, lane, kdim, vec, live);
        }
      if (c == lo) first();
#pragma unroll
      for (int s = 0; s < D; ++s)
        if (c + s < hi) {
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            k[s].w[j].s = sc[j].block(s);
            acc[j] = mma_planes<FMT, 1>(k[s].x, k[s].w[j], lane, acc[j]);
          }
        }
    }
    if (hi <= lo) first();
  }
}

// A gate/up tile: the first 8 rows lie in the gate matrix of an expert, the others in
// its up matrix.
template <int FMT>
__device__ __forceinline__ Matrices gate_up(const void* wg, const void* wu, const void* sg, const void* su, int expert,
                                            int width, int H) {
  const size_t w = static_cast<size_t>(expert) * width * row_bytes<FMT>(H);
  const size_t s = static_cast<size_t>(expert) * width * scale_bytes<FMT>(H);
  return Matrices{{static_cast<const uint8_t*>(wg) + w, static_cast<const uint8_t*>(wu) + w},
                  {static_cast<const uint8_t*>(sg) + s, static_cast<const uint8_t*>(su) + s}};
}
// Its columns [n0, n0 + 8) (past the width: the last row again, not stored).
template <int FMT>
__device__ __forceinline__ WRow gate_up_row(const Matrices& m, int n0, int width, int H, int lane) {
  const int row = min(n0 + (lane & 7), width - 1);
  return weight_rows<FMT>(m, row, row, H, lane);
}

// A store that other workgroups of the running kernel may read: written through to
// the memory that the eight L2 caches share, so that making it visible needs no
// write-back of a whole cache.
template <class V>
__device__ __forceinline__ void st_shared(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A load of what st_shared stored, from the same memory.
template <class V>
__device__ __forceinline__ V ld_shared(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// This wave's stores have reached that memory.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

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
    const float h = s[i] / (1.0f + expf(-s[i])) * up;
    const size_t o = base + static_cast<size_t>(max(row, 0)) * width + n0 + r;
    if constexpr (FMT == kDtypeF32) {
      if (r < 8 && n0 + r < width && row >= 0) st_shared(static_cast<float*>(a.h[0]) + o, h);
    } else {
      // What a plane leaves over goes to the next; an infinite plane leaves nothing
      // (inf - inf would turn it into NaN).  Widths are even, lanes store in pairs.
      float rest = h;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const uint32_t b = f32_to_bf16_bits(rest);
        const float v = bf16_bits_to_f32(static_cast<uint16_t>(b));
        rest = fabsf(v) < INFINITY ? rest - v : 0.f;
        const uint32_t pair = b | (__shfl_xor(b, 1, kWave) << 16);
        if (r < 8 && !(r & 1) && row >= 0) st_shared(reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.h[p]) + o), pair);
      }
    }
  }
}

// Counters in the workspace, cleared by the first kernel; each on a line of its own
// (atomics on one line take about 10 ns each, whoever sends them).
struct Ctl {
  static constexpr int kLine = 32;                          // ints
  static constexpr int kQueue = 0;                          // next gate/up item of each queue
  static constexpr int kSharedQueue = kQueue + kQueues * kLine;   // the same for the shared expert
  static constexpr int kDone = kSharedQueue + kQueues * kLine;    // finished tiles, in 16 counters
  static constexpr int kGroups = 16;
  static constexpr int kGo = kDone + kGroups * kLine;       // all tiles finished, one flag for each group
  static constexpr int kRange = kGo + kGroups * kLine;      // next down range
  static constexpr int kRouted = kRange + kLine;            // routing published, one flag for four tokens
  static constexpr int kTile = kRouted + 4 * kLine;         // finished parts of each down tile
};
__host__ __device__ inline int ctl_ints(int H) { return Ctl::kTile + (H + 15) / 16; }   // enough for any kSets

__device__ __forceinline__ int ctl_add(int* p, int v) {
  return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- first kernel

__host__ __device__ inline int router_tiles(int E, int S) { return (E + 15) / 16 + (S > 0 ? 1 : 0); }

// AFMT: the type of x and of the router.
template <int AFMT>
__global__ void __launch_bounds__(kFewThreads, 2) few_first_kernel(FewArgs a) {
  __shared__ Red red;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  for (int i = blockIdx.x * kFewThreads + tid; i < ctl_ints(a.H); i += gridDim.x * kFewThreads) a.ctl[i] = 0;

  const uint32_t xoff = static_cast<uint32_t>(min(r, a.T - 1)) * static_cast<uint32_t>(row_bytes<AFMT>(a.H));
  // 16 logits; the last tile is the shared gate's, alone in a matrix of one row.
  const int part = blockIdx.x % a.parts, tile = blockIdx.x / a.parts;
  const int nb = static_cast<int>(ceil_div(a.H, SkinnyFmt<AFMT>::kBlk));
  const bool gate = tile * 16 >= a.E;
  const int c0 = gate ? a.E : tile * 16, cols = gate ? 1 : min(16, a.E - c0);
  const void* w = gate ? a.w_gcol : a.w_router;
  const Matrices m{{w, w}, {nullptr, nullptr}};
  const int row0 = (gate ? 0 : c0) + min(lane & 7, cols - 1), row1 = (gate ? 0 : c0) + min(8 + (lane & 7), cols - 1);
  const WRow row[1] = {weight_rows<AFMT>(m, row0, row1, a.H, lane)};
  f32x4 acc[1];
  wave_tiles<AFMT, 1>(m, row, a.x, xoff, r < a.T, part * nb / a.parts, (part + 1) * nb / a.parts, a.H, a.hvec, wave,
                      lane, acc, [] {});
  red.v[wave][lane] = acc[0];
  __syncthreads();
  if (wave == 0 && r < cols) {
    const f32x4 s = red_sum(red, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a.z[(static_cast<size_t>(part) * kFewTokens + 4 * g + i) * a.ldz + c0 + r] = s[i];
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

// Maximum over the wave: rotations within the rows of 16 lanes, then the four rows.
template <int CTRL>
__device__ __forceinline__ uint32_t ror_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = ror_max<0x121>(v);
  v = ror_max<0x122>(v);
  v = ror_max<0x124>(v);
  v = ror_max<0x128>(v);
  const int i = static_cast<int>(v);
  const uint32_t a = static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 0)), b = static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 16)),
                 c = static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 32)), d = static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 48));
  return max(max(a, b), max(c, d));
}

// Looks at the routing flags before a workgroup does the routing itself (0.4 us each or
// more).
constexpr int kRouteTries = 64;

constexpr double kFewFixed = 8589934592.0;   // 2^33: budget aggregates in fixed point, as in moe_route

// What every workgroup knows of the call's routing.
struct Routing {
  int ids[kFewSlots];              // [T, K]
  float w[kFewSlots];
  float sg[kFewTokens];            // sigmoid of the shared gate
  int n;                           // touched experts
  int seg_expert[kFewSlots];
  int16_t seg_slot[kFewSlots + 1][kFewTokens];   // row of h of (segment, token), -1: not served
  alignas(16) float seg_w[kFewSlots + 1][kFewTokens];   // its weight, 0 if not served
};
static_assert(offsetof(Routing, seg_w) % 16 == 0 && alignof(Routing) >= 16, "seg_w is read four floats at a time");
struct RouteScratch {
  unsigned long long agg[kMaxExperts];
  int seg_of[kMaxExperts];
  int nu, dropped, empty;
  struct alignas(16) {
    unsigned long long mass;
    int id;
  } list[kFewSlots];               // the experts in use
};

// Top-k of token t by one wave (same selection and trim as moe_route).  A lane holds
// the keys of experts 4 lane .. + 4 (and 256 further on), sorted; each round takes the
// largest head of the lanes.
template <int NQ>
__device__ __forceinline__ void route_token(const FewArgs& a, Routing& R, int t, int lane) {
  constexpr int NJ = 4 * NQ;
  const size_t plane = static_cast<size_t>(kFewTokens) * a.ldz;
  const float* zr = a.z + static_cast<size_t>(t) * a.ldz;
  const float* bias = a.bias ? a.bias + static_cast<size_t>(t) * a.E : nullptr;
  uint32_t key[NJ];
  int id[NJ];
  // All loads first.  Rows of z are multiples of 16 long; a lane takes 4 columns at a time.
  f32x4 v[NQ][kFewRouterParts];
  float b[NJ], gv[kFewRouterParts];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = 4 * (lane + kWave * q);
#pragma unroll
    for (int p = 0; p < kFewRouterParts; ++p)
      v[q][p] = p < a.parts && e < a.E ? *reinterpret_cast<const f32x4*>(zr + p * plane + e) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) b[4 * q + c] = bias && e + c < a.E ? bias[e + c] : 0.f;
  }
#pragma unroll
  for (int p = 0; p < kFewRouterParts; ++p) gv[p] = p < a.parts && a.S > 0 ? zr[p * plane + a.E] : 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int e = 4 * (lane + kWave * (j / 4)) + j % 4;
    float z = v[j / 4][0][j % 4];
#pragma unroll
    for (int p = 1; p < kFewRouterParts; ++p) z += v[j / 4][p][j % 4];
    z += b[j];
    key[j] = e < a.E ? order_key(z == z ? z : -INFINITY) : 0;
    id[j] = e;
  }
  float gate = gv[0];
#pragma unroll
  for (int p = 1; p < kFewRouterParts; ++p) gate += gv[p];
  // Odd-even merge sort of 4 or 8: descending, the lower id first among equals.
  auto order = [&](int x, int y) __attribute__((always_inline)) {
    const bool swap = key[y] > key[x] || (key[y] == key[x] && id[y] < id[x]);
    const uint32_t k = swap ? key[y] : key[x];
    key[y] = swap ? key[x] : key[y];
    key[x] = k;
    const int e = swap ? id[y] : id[x];
    id[y] = swap ? id[x] : id[y];
    id[x] = e;
  };
  order(0, 1); order(2, 3); order(0, 2); order(1, 3); order(1, 2);
  if constexpr (NJ > 4) {
    order(4, 5); order(6, 7); order(4, 6); order(5, 7); order(5, 6);
    order(0, 4); order(1, 5); order(2, 6); order(3, 7); order(2, 4); order(3, 5); order(1, 2); order(3, 4); order(5, 6);
  }
  const float zmax = key_value(wave_max_u32(key[0]));
  // Softmax denominator over all experts (only without renormalisation).
  float denom_all = 0.f;
  if (!a.norm) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (key[j] != 0) denom_all += expf(key_value(key[j]) - zmax);
    denom_all = wave_sum(denom_all);
  }
  int my_id = -1;
  float my_z = 0.f;
  for (int k = 0; k < a.K; ++k) {
    const uint32_t m = wave_max_u32(key[0]);
    unsigned long long has = __ballot(key[0] == m);
    int owner = __builtin_ctzll(has), e = __builtin_amdgcn_readlane(id[0], owner);
    for (has &= has - 1; has; has &= has - 1) {        // ties: the lowest id
      const int o = __builtin_ctzll(has), f = __builtin_amdgcn_readlane(id[0], o);
      if (f < e) { e = f; owner = o; }
    }
    const bool pop = lane == owner;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      key[j] = pop ? (j + 1 < NJ ? key[j + 1 < NJ ? j + 1 : j] : 0) : key[j];
      id[j] = pop ? id[j + 1 < NJ ? j + 1 : j] : id[j];
    }
    if (lane == k) { my_id = e; my_z = key_value(m); }
  }
  const float p = lane < a.K ? expf(my_z - zmax) : 0.f;
  bool kept = lane < a.K;
  if (a.top_p > 0.f) {
    float before = 0.f, all = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const float pk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), k));
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
  if (lane == 0) R.sg[t] = a.S > 0 ? 1.0f / (1.0f + expf(-gate)) : 0.f;
}

__device__ __forceinline__ void route_token_any(const FewArgs& a, Routing& R, int t, int lane) {
  if (a.E <= 256) route_token<1>(a, R, t, lane);
  else route_token<2>(a, R, t, lane);
}

// Routes and publishes tokens 4 j to 4 j + 3 (j: the workgroup).
__device__ __forceinline__ void publish_routing(const FewArgs& a, Routing& R, int j, int wave, int lane) {
  const int tid = threadIdx.x, t = j * kFewWaves + wave;
  if (t < a.T) route_token_any(a, R, t, lane);
  __syncthreads();
  const int first = j * kFewWaves * a.K, n = min(kFewWaves * a.K, a.T * a.K - first);
  if (tid < n) {
    st_shared(a.routed + first + tid, R.ids[first + tid]);
    st_shared(a.routed + kFewSlots + first + tid, __float_as_int(R.w[first + tid]));
  }
  if (tid < kFewWaves && j * kFewWaves + tid < a.T)
    st_shared(a.routed + 2 * kFewSlots + j * kFewWaves + tid, __float_as_int(R.sg[j * kFewWaves + tid]));
  stores_done();
  __syncthreads();
  if (tid == 0) st_shared(a.ctl + Ctl::kRouted + j * Ctl::kLine, 1);
}

// All tokens' routing.  Up to a token for each wave, worked out here; more, as published,
// or if that does not come in time, here too.
__device__ __forceinline__ void fetch_routing(const FewArgs& a, Routing& R, RouteScratch& C, int wave, int lane) {
  const int tid = threadIdx.x, groups = (a.T + kFewWaves - 1) / kFewWaves;
  if (wave == 0) {
    bool there = false;
    for (int i = 0; i < kRouteTries && !there && groups > 1; ++i) {
      if (i > 0) __builtin_amdgcn_s_sleep(4);
      there = __all(lane >= groups || ld_shared(a.ctl + Ctl::kRouted + min(lane, groups - 1) * Ctl::kLine) != 0);
    }
    if (lane == 0) C.nu = there;
  }
  __syncthreads();
  if (C.nu) {
    if (tid < a.T * a.K) {
      R.ids[tid] = ld_shared(a.routed + tid);
      R.w[tid] = __int_as_float(ld_shared(a.routed + kFewSlots + tid));
    }
    if (tid < a.T) R.sg[tid] = __int_as_float(ld_shared(a.routed + 2 * kFewSlots + tid));
  } else {
    for (int t = wave; t < a.T; t += kFewWaves) route_token_any(a, R, t, lane);
  }
  __syncthreads();
}

// The budget over all tokens, as in moe_route, then the touched experts' segments.
__device__ __forceinline__ void finish_routing(const FewArgs& a, Routing& R, RouteScratch& C, bool report) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
        if (atomicExch(&C.seg_of[e], 1) == 0) C.list[atomicAdd(&C.nu, 1)].id = e;
      }
    }
    __syncthreads();
    const int nu = C.nu;
    const bool active = a.budget > 0 && nu > a.budget;
    if (active) {
      int e = -1, rank = 0;
      unsigned long long mass = 0;
      if (tid < nu) {
        e = C.list[tid].id;
        mass = C.list[tid].mass = C.agg[e];
      }
      __syncthreads();
#pragma unroll 4
      for (int o = 0; o < nu; ++o) {
        const auto other = C.list[o];
        rank += static_cast<int>(other.mass > mass) | (static_cast<int>(other.mass == mass) & static_cast<int>(other.id < e));
      }
      __syncthreads();
      if (e >= 0) C.seg_of[e] = rank < a.budget ? 1 : 0;
      __syncthreads();
      // Kept slots to the front, a wave for each token.
      for (int t = wave; t < a.T; t += kFewWaves) {
        int* ir = R.ids + t * a.K;
        float* wr = R.w + t * a.K;
        const int id = lane < a.K ? ir[lane] : -1;
        const float w = lane < a.K ? wr[lane] : 0.f;
        const bool keep = id >= 0 && C.seg_of[id] != 0;
        const unsigned long long kept = __ballot(keep), dropped = __ballot(id >= 0 && !keep);
        const int nk = __popcll(kept);
        if (dropped) {
          const float sum = wave_sum(keep ? w : 0.f);
          if (lane < a.K && lane >= nk) { ir[lane] = -1; wr[lane] = 0.f; }
          if (keep) {
            const int at = __popcll(kept & ((1ull << lane) - 1));
            ir[at] = id;
            wr[at] = a.norm && sum != 0.f ? w / sum : w;   // only weights of 0: they stay
          }
          if (lane == 0) atomicAdd(&C.dropped, __popcll(dropped));
        }
        if (nk == 0 && lane == 0) atomicAdd(&C.empty, 1);
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
  for (int i = tid; i < (R.n + 1) * kFewTokens; i += kFewThreads) {
    (&R.seg_slot[0][0])[i] = -1;
    (&R.seg_w[0][0])[i] = 0.f;
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

// A block of the down half: weights and the planes of h that meet them.
template <int FMT>
struct DownBlk {
  static constexpr int kPlanes = FMT == kDtypeF32 ? 1 : 3;
  WBlk<FMT> w[FewBatch<FMT>::kSets];
  XBlk<FMT> h[kPlanes];
};

// The next gate/up item, or -1 when all queues are empty (called by one thread; all
// queues from `home` on are tried, `tried` of them have been found empty).  Queue q
// holds the q-th eighth of the items.
__device__ __forceinline__ int take_item(int* queues, int items, int home, int& tried) {
  for (; tried < kQueues; ++tried) {
    const int q = (home + tried) % kQueues;
    const int lo = q * items / kQueues, n = (q + 1) * items / kQueues - lo;
    int* c = queues + q * Ctl::kLine;
    // Other queues are looked at before they are written to.
    if (tried > 0 && ld_shared(c) >= n) continue;
    const int i = ctl_add(c, 1);
    if (i < n) return lo + i;
  }
  return -1;
}

// The down half: the output tiles (16 kSets columns), each contracted over the blocks of all
// touched experts and the shared expert, are one line of tiles * nblk blocks that is
// cut into equal ranges, so that every workgroup reads the same number of weights.
// A tile that a cut goes through is added up from its parts, in their order, by the
// workgroup that finishes its part last.
// Short lines are cut into one range for each workgroup (or fewer).  Long ones are cut
// into a range of half that length for each, then as many of a quarter, then twice as
// many of an eighth, which are handed out as ranges are finished: few parts, and a
// short last one.
constexpr int kMaxRanges = 4 * kFewGrid;
constexpr int kShortRange = 2 * kFewWaves;   // blocks: two for each wave
constexpr int kLongRange = 16 * kFewWaves;
constexpr int kPartsAhead = 4;               // parts of a tile read at a time
struct DownCut {
  int tiles, nblk, ranges, q, rem;
  bool graded;
  __device__ __forceinline__ DownCut(int tiles_, int nblk_) : tiles(tiles_), nblk(nblk_) {
    const int all = tiles * nblk;
    graded = all >= kLongRange * kFewGrid;
    // In units of q blocks: ungraded ranges are one unit, the graded ones 4, 2 and 1.
    const int units = graded ? 8 * kFewGrid : max(1, min(kFewGrid, all / kShortRange));
    ranges = graded ? kMaxRanges : units;
    q = all / units;
    rem = all - q * units;                     // the first rem units are one block longer
  }
  __device__ __forceinline__ int unit_start(int u) const { return u * q + min(u, rem); }
  __device__ __forceinline__ int start(int b) const {
    if (!graded) return unit_start(b);
    return unit_start(b <= kFewGrid ? 4 * b : b <= 2 * kFewGrid ? 2 * (b + kFewGrid) : b + 4 * kFewGrid);
  }
  __device__ __forceinline__ int owner(int f) const {          // the range that holds block f
    const int longer = rem * (q + 1);
    const int u = f < longer ? f / (q + 1) : rem + (f - longer) / q;
    if (!graded) return u;
    return u < 4 * kFewGrid ? u / 4 : u < 6 * kFewGrid ? u / 2 - kFewGrid : u - 4 * kFewGrid;
  }
};

// This workgroup's gate/up items of NS tiles each: `shared_items` of the shared expert
// first, then `tiles` for each touched expert, handed out from the queues; returns how
// many it ran.  The next item is taken while one is running, but not before the first
// loads are on their way: a workgroup that comes early must not take the only item of
// one that comes late.
enum class Items { Shared, Routed, Both };
template <int FMT, int NS, Items KIND>
__device__ __forceinline__ int gate_up_half(const FewArgs& a, const Routing& R, Red* red, int& s_next, int* queues,
                                            int shared_items, int items, int tiles, int wave, int lane) {
  using F = SkinnyFmt<FMT>;
  const int r = lane & 15, hb = static_cast<int>(ceil_div(a.H, F::kBlk));
  const uint32_t xoff = static_cast<uint32_t>(min(r, a.T - 1)) * static_cast<uint32_t>(a.H) * (F::kF32 ? 4 : 2);
  const int tid = threadIdx.x, home = blockIdx.x % kQueues;
  int tried = 0, finished = 0;
  // Workgroups 0 to 255 lie on different CUs.  If there is no more than one item for
  // each CU the others come two microseconds later, so that no CU runs two: 24.4 us instead
  // of 25.9 (8 experts, top-2, I 512, shared 512, H 2048, 1 token, bf16), 112.1 instead of
  // 113.6 (512 experts, fp8, 5 tokens), elsewhere within 1 % of each other.
  if (items <= kFewGrid / 2 && blockIdx.x >= kFewGrid / 2) __builtin_amdgcn_s_sleep(64);
  if (tid == 0) s_next = take_item(queues, items, home, tried);
  __syncthreads();
  int item = __builtin_amdgcn_readfirstlane(s_next);
  while (item >= 0) {
    const bool shared = KIND == Items::Shared || (KIND == Items::Both && item < shared_items);
    const int routed = KIND == Items::Routed ? item : item - shared_items, seg = shared ? 0 : routed / tiles;
    const int n0 = (shared ? item : routed - seg * tiles) * (8 * NS), width = shared ? a.S : a.I;
    const int e = shared ? 0 : __builtin_amdgcn_readfirstlane(R.seg_expert[seg]);
    const Matrices m = gate_up<FMT>(shared ? a.ws_gate : a.w_gate, shared ? a.ws_up : a.w_up,
                                    shared ? a.ss_gate : a.s_gate, shared ? a.ss_up : a.s_up, e, width, a.H);
    WRow row[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) row[j] = gate_up_row<FMT>(m, n0 + 8 * j, width, a.H, lane);
    int next = -1;
    f32x4 acc[NS];
    wave_tiles<FMT, NS>(m, row, a.x, xoff, shared ? r < a.T : R.seg_slot[seg][r] >= 0, 0, hb, a.H, a.hvec, wave, lane,
                        acc, [&]() __attribute__((always_inline)) {
                          if (tid == 0) next = take_item(queues, items, home, tried);
                        });
    __syncthreads();                 // s_next has been read, the previous tiles added up
#pragma unroll
    for (int j = 0; j < NS; ++j) red[j].v[wave][lane] = acc[j];
    if (tid == 0) s_next = next;
    __syncthreads();
    item = __builtin_amdgcn_readfirstlane(s_next);
    if (wave == 0) {
      const size_t base = shared ? static_cast<size_t>(a.T) * a.K * a.I : 0;
#pragma unroll
      for (int j = 0; j < NS; ++j)
        store_h<FMT>(a, red_sum(red[j], lane), base, n0 + 8 * j, width, lane, [&](int t) __attribute__((always_inline)) {
          return shared ? (t < a.T ? t : -1) : static_cast<int>(R.seg_slot[seg][t]);
        });
    }
    ++finished;
  }
  __syncthreads();                   // red and s_next are free
  return finished;
}

template <int FMT>
__global__ void __launch_bounds__(kFewThreads, 2) few_second_kernel(FewArgs a) {
  using F = SkinnyFmt<FMT>;
  constexpr int NS = FewBatch<FMT>::kSets, kWide = FewBatch<FMT>::kWide;
  // The routing's scratch is done with when the first tile is added up.
  __shared__ union {
    RouteScratch scratch;
    Red red[kMaxSets];
  } U;
  __shared__ Routing R;
  Red* const red = U.red;
  __shared__ int s_next, s_ready;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  if (tid == 0) s_ready = 0;
  // ---- the gate/up half.  Up to four tokens are routed by every workgroup at once,
  // before the memory is busy, and all items are handed out together.  More tokens are
  // routed by a few workgroups while the others run the shared expert's items.
  const bool few = a.T <= kFewWaves;
  const int shared_items = static_cast<int>(ceil_div(a.S, 8));
  int finished = 0;
  if (!few) {
    if (static_cast<int>(blockIdx.x) * kFewWaves < a.T) publish_routing(a, R, blockIdx.x, wave, lane);
    if (a.S > 0)
      finished = gate_up_half<FMT, 1, Items::Shared>(a, R, red, s_next, a.ctl + Ctl::kSharedQueue, shared_items,
                                                     shared_items, 1, wave, lane);
  }
  fetch_routing(a, R, U.scratch, wave, lane);
  finish_routing(a, R, U.scratch, blockIdx.x == 0);
  const int n = R.n;
  int tiles = static_cast<int>(ceil_div(a.I, 8));
  if (kWide > 1 && !few && n * tiles >= kWideTiles * kFewGrid) {
    tiles = static_cast<int>(ceil_div(a.I, 8 * kWide));
    finished += gate_up_half<FMT, kWide, Items::Routed>(a, R, red, s_next, a.ctl + Ctl::kQueue, 0, n * tiles, tiles,
                                                        wave, lane);
  } else {
    const int first = few ? shared_items : 0;
    finished += gate_up_half<FMT, 1, Items::Both>(a, R, red, s_next, a.ctl + Ctl::kQueue, first, first + n * tiles,
                                                  tiles, wave, lane);
  }
  const int items = shared_items + n * tiles;
  // Every h of this workgroup was stored by wave 0.  The last one to count sees all
  // counts, and says so to the others: polling the counters themselves slowed those
  // who still had to count.
  int* go = a.ctl + Ctl::kGo;
  auto all_counted = [&]() {
    int c = lane < Ctl::kGroups ? ld_shared(a.ctl + Ctl::kDone + lane * Ctl::kLine) : 0;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) c += __shfl_xor(c, o, 16);
    return __builtin_amdgcn_readfirstlane(c) >= items;
  };
  const int group = blockIdx.x % Ctl::kGroups;
  if (wave == 0 && finished > 0) {
    stores_done();
    if (lane == 0) ctl_add(a.ctl + Ctl::kDone + group * Ctl::kLine, finished);
    stores_done();
    if (all_counted() && lane < Ctl::kGroups) st_shared(go + lane * Ctl::kLine, 1);
  }

  // ---- the down half
  const int ib = static_cast<int>(ceil_div(a.I, F::kBlk)), sb = static_cast<int>(ceil_div(a.S, F::kBlk));
  const int nblk = n * ib + sb;
  if (nblk == 0) {                   // no expert at all: y is zero
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kFewThreads + tid; i < static_cast<int64_t>(a.T) * a.H;
         i += kFewGrid * kFewThreads) {
      if (a.y) a.y[i] = 0.f;
      if (a.y_act) {
        if (a.act_bf16) static_cast<uint16_t*>(a.y_act)[i] = 0;
        else static_cast<float*>(a.y_act)[i] = 0.f;
      }
    }
    return;
  }
  const DownCut cut(static_cast<int>(ceil_div(a.H, 16 * NS)), nblk);
  if (blockIdx.x >= cut.ranges) return;
  // Waits until every h is there: wave 0 for the grid, the others for wave 0.  Only
  // wave 0 invalidates the caches (for the whole CU and its L2); when all waves did,
  // that took 10 us.
  bool ready = false;
  auto wait_for_h = [&]() __attribute__((always_inline)) {
    if (ready) return;
    ready = true;
    if (wave == 0) {
      // The flag is one line for 32 workgroups; now and then the counts themselves.
      if (items > 0)
        for (int i = 1; ld_shared(go + group * Ctl::kLine) == 0; ++i) {
          if (i % 16 == 0 && all_counted()) break;
          __builtin_amdgcn_s_sleep(8);
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      __hip_atomic_store(&s_ready, 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
    } else {
      while (__hip_atomic_load(&s_ready, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) == 0) __builtin_amdgcn_s_sleep(4);
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    }
  };
  const size_t h_shared = static_cast<size_t>(a.T) * a.K * a.I;
  int b = blockIdx.x;
  while (b < cut.ranges) {
    const int f0 = cut.start(b), f1 = cut.start(b + 1);
    const int tile0 = f0 / nblk, tile1 = (f1 - 1) / nblk;
    int next = cut.ranges;
    if (tid == 0 && cut.ranges > kFewGrid) next = kFewGrid + ctl_add(a.ctl + Ctl::kRange, 1);
    for (int tile = tile0; tile <= tile1; ++tile) {
      const int base = tile * nblk;
      const int k0 = max(f0 - base, 0), k1 = min(f1 - base, nblk);
      const int lo = k0 + wave * (k1 - k0) / kFewWaves, hi = k0 + (wave + 1) * (k1 - k0) / kFewWaves;
      // Positions of the weights' loads, of h's loads and of their use: expert segment
      // and block in it.
      struct Pos {
        int seg, kb;
      };
      const int seg0 = min(lo / ib, n);
      Pos lw{seg0, lo - seg0 * ib}, lh = lw, u = lw;
      // Whether a new segment begins.
      auto step = [&](Pos& p) __attribute__((always_inline)) {
        if (p.seg == n || ++p.kb < ib) {
          p.kb += p.seg == n;
          return false;
        }
        ++p.seg;
        p.kb = 0;
        return true;
      };
      Matrices m{};
      WRow row[NS];
      auto enter_w = [&]() __attribute__((always_inline)) {
        const bool shared = lw.seg == n;
        const int width = (shared ? a.S : a.I);
        const size_t first = shared ? 0 : static_cast<size_t>(__builtin_amdgcn_readfirstlane(R.seg_expert[lw.seg])) * a.H;
        m.w[0] = m.w[1] = static_cast<const uint8_t*>((shared ? a.ws_down : a.w_down)) + first * row_bytes<FMT>(width);
        m.s[0] = m.s[1] = static_cast<const uint8_t*>((shared ? a.ss_down : a.s_down)) + first * scale_bytes<FMT>(width);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int row0 = (tile * NS + j) * 16 + (lane & 7);
          row[j] = weight_rows<FMT>(m, min(row0, a.H - 1), min(row0 + 8, a.H - 1), width, lane);
        }
      };
      uint32_t hoff = 0;
      size_t hbase = 0;
      bool live = false;
      auto enter_h = [&]() __attribute__((always_inline)) {
        const bool shared = lh.seg == n;
        const int slot = R.seg_slot[lh.seg][r];
        live = slot >= 0;
        hbase = (shared ? h_shared : 0) * (F::kF32 ? 4 : 2);
        hoff = static_cast<uint32_t>(max(slot, 0)) * static_cast<uint32_t>((shared ? a.S : a.I)) * (F::kF32 ? 4 : 2);
      };
      if (lo < hi) {
        enter_w();
        enter_h();
      }
      f32x4 acc[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      constexpr int D = FewBatch<FMT>::kDown, DS = FewBatch<FMT>::kDownScales;
      Scales<FMT, DS> sc[NS];        // of the coming blocks, `scales` of them
      int scales = 0;
      for (int c = lo; c < hi; c += D) {
        DownBlk<FMT> k[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
          if (c + d < hi) {
            const bool shared = lw.seg == n;
#pragma unroll
            for (int j = 0; j < NS; ++j)
              load_w<FMT>(k[d].w[j], m, row[j], lw.kb, lane, (shared ? a.S : a.I), (shared ? a.svec : a.ivec));
            if constexpr (Scales<FMT, 1>::kAny) {
              static_assert(D == 1, "one block's scales at a time");
              if (scales == 0) {
                const int left = (shared ? sb : ib) - lw.kb;
                scales = min(left, DS);
#pragma unroll
                for (int j = 0; j < NS; ++j) sc[j].load(row[j].s + blk_scale_bytes<FMT>() * lw.kb, left);
              }
              --scales;
            }
            if (step(lw) && c + d + 1 < hi) enter_w();
          }
        // The weights do not depend on h: the first ones are on their way during the wait.
        wait_for_h();
#pragma unroll
        for (int d = 0; d < D; ++d)
          if (c + d < hi) {
            const bool shared = lh.seg == n;
#pragma unroll
            for (int p = 0; p < DownBlk<FMT>::kPlanes; ++p)
              load_x<FMT>(k[d].h[p], static_cast<const uint8_t*>(a.h[p]) + hbase, hoff, lh.kb, lane,
                          (shared ? a.S : a.I), (shared ? a.svec : a.ivec), live);
            if (step(lh) && c + d + 1 < hi) enter_h();
          }
#pragma unroll
        for (int d = 0; d < D; ++d)
          if (c + d < hi) {
            const float4 wt = *reinterpret_cast<const float4*>(&R.seg_w[u.seg][4 * g]);
            const float ws[4] = {wt.x, wt.y, wt.z, wt.w};
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              k[d].w[j].s = sc[j].block(0);
              sc[j].step();
              const f32x4 t = mma_planes<FMT, DownBlk<FMT>::kPlanes>(k[d].h, k[d].w[j], lane, f32x4{0.f, 0.f, 0.f, 0.f});
              // A token that the expert does not serve takes nothing, not 0 * inf either.
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[j][q] = ws[q] != 0.f ? fmaf(ws[q], t[q], acc[j][q]) : acc[j][q];
            }
            step(u);
          }
      }
      wait_for_h();                  // a wave without a block
      __syncthreads();               // the previous tile has been added up
#pragma unroll
      for (int j = 0; j < NS; ++j) red[j].v[wave][lane] = acc[j];
      if (tid == 0) s_next = next;
      __syncthreads();
      if (wave != 0) continue;
      f32x4 s[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) s[j] = red_sum(red[j], lane);
      if (k0 > 0 || k1 < nblk) {     // a part: the last one to arrive adds them up
        const int b0 = cut.owner(base), b1 = cut.owner(base + nblk - 1);
        float* part = a.part + (static_cast<size_t>(b) * 2 + (tile == tile0 ? 0 : 1)) * (256 * NS);
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) st_shared(part + 256 * j + 64 * i + lane, s[j][i]);
        stores_done();
        int before = 0;
        if (lane == 0) before = ctl_add(a.ctl + Ctl::kTile + tile, 1);
        if (__builtin_amdgcn_readfirstlane(before) != b1 - b0) continue;
#pragma unroll
        for (int j = 0; j < NS; ++j) s[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int o = b0; o <= b1; o += kPartsAhead) {
          float v[kPartsAhead][NS][4];
#pragma unroll
          for (int d = 0; d < kPartsAhead; ++d) {
            // The tile is range o's first one, unless the range began in an earlier tile.
            const int at = min(o + d, b1);
            const float* p = a.part + (static_cast<size_t>(at) * 2 + (cut.start(at) / nblk == tile ? 0 : 1)) * (256 * NS);
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) v[d][j][i] = ld_shared(p + 256 * j + 64 * i + lane);
          }
#pragma unroll
          for (int d = 0; d < kPartsAhead; ++d)
            if (o + d <= b1)
#pragma unroll
              for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] += v[d][j][i];
        }
      }
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int col = (tile * NS + j) * 16 + r;
        if (col >= a.H) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 4 * g + i;
          if (t < a.T) {
            const size_t o = static_cast<size_t>(t) * a.H + col;
            if (a.y) a.y[o] = s[j][i];
            if (a.y_act) {
              if (a.act_bf16) static_cast<uint16_t*>(a.y_act)[o] = f32_to_bf16_bits(s[j][i]);
              else static_cast<float*>(a.y_act)[o] = s[j][i];
            }
          }
        }
      }
    }
    b = __builtin_amdgcn_readfirstlane(s_next);
  }
}

// ---------------------------------------------------------------- host

struct FewLayout {
  size_t ctl, z, h[3], routed, part, total;
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
  // Parts of one batch of each wave.
  const int blocks = static_cast<int>(ceil_div(c.hidden_size, f32 ? 32 : 64));
  L.parts = static_cast<int>(std::min<int64_t>(kFewRouterParts, ceil_div(blocks, 10 * kFewWaves)));
  L.ctl = take(ctl_ints(c.hidden_size) * sizeof(int));
  L.z = take(static_cast<size_t>(L.parts) * kFewTokens * L.ldz * sizeof(float));
  const size_t elems = static_cast<size_t>(T) * c.num_experts_per_tok * c.moe_intermediate_size +
                       static_cast<size_t>(T) * c.shared_expert_intermediate_size;
  for (int p = 0; p < 3; ++p) L.h[p] = take(f32 ? (p ? 0 : elems * 4) : elems * 2);
  L.routed = take((2 * kFewSlots + kFewTokens) * sizeof(int));
  L.part = take(static_cast<size_t>(kMaxRanges) * 2 * kMaxSets * 256 * sizeof(float));
  L.total = off;
  return L;
}

// The second kernel numbers its gate/up tiles and its down blocks in 32 bits; offsets
// within x, one expert's matrix and a plane of h are 32-bit byte offsets.
bool few_countable(const moe_config& c, int64_t T) {
  const int64_t experts = std::min<int64_t>(c.n_routed_experts, kFewSlots);
  const int64_t H = c.hidden_size, I = c.moe_intermediate_size, S = c.shared_expert_intermediate_size;
  const int64_t nblk = experts * ceil_div(I, 32) + ceil_div(S, 32), lim = int64_t{1} << 31;
  const int64_t size = c.weight_dtype == MOE_DTYPE_F32 ? 4 : 2;
  return (experts * ceil_div(I, 8) + ceil_div(S, 8)) * kQueues < lim && ceil_div(H, 16) * nblk < lim && T * H * size < 2 * lim &&
         H * I * size < 2 * lim && H * S * size < 2 * lim && H * c.n_routed_experts * size < 2 * lim &&
         (kFewSlots * I + kFewTokens * S) * size < 2 * lim;
}

bool misaligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <int FMT>
int few_launch(const FewArgs& a, hipStream_t s) {
  constexpr int AFMT = FMT == kDtypeF32 ? kDtypeF32 : kDtypeBf16;
  few_first_kernel<AFMT><<<router_tiles(a.E, a.S) * a.parts, kFewThreads, 0, s>>>(a);
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
  if (max_tokens > kFewTokens || !few_countable(*cfg, max_tokens)) return MOE_ERR_UNSUPPORTED;
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
  for (int p = 0; p < 3; ++p) a.h[p] = ws + L.h[p];
  a.routed = reinterpret_cast<int*>(ws + L.routed);
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.T = T;
  a.H = cfg->hidden_size;
  a.E = cfg->n_routed_experts;
  a.I = cfg->moe_intermediate_size;
  a.K = cfg->num_experts_per_tok;
  a.S = cfg->shared_expert_intermediate_size;
  a.ldz = L.ldz;
  a.parts = L.parts;
  a.norm = cfg->norm_topk_prob;
  a.budget = cfg->expert_budget;
  a.top_p = (cfg->top_p > 0.f && cfg->top_p < 1.f) ? cfg->top_p : 0.f;
  a.hvec = wide && a.H % 4 == 0;
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
