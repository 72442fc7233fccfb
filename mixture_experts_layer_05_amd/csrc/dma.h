// Loads from memory straight into LDS, and the waits for them (included by the kernels
// that use them).
#pragma once

#include "common.h"

namespace moe {
namespace {

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p));
}

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Buffer resource words for a raw byte buffer.
__device__ __forceinline__ i32x4_t dma_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  i32x4_t r = {static_cast<int>(static_cast<uint32_t>(p)), static_cast<int>(static_cast<uint32_t>(p >> 32) & 0xffff),
               static_cast<int>(bytes), 0x00020000};
  r.x = __builtin_amdgcn_readfirstlane(r.x);
  r.y = __builtin_amdgcn_readfirstlane(r.y);
  r.z = __builtin_amdgcn_readfirstlane(r.z);
  return r;
}

// Wave instructions of buffer loads with the LDS flag.  Instruction q: lane l
// loads 16 bytes at resource offset voff[q] + soff and writes them to LDS at
// lds + 1024 q + 16 l (M0 holds the LDS address; a write of M0 needs one wait
// state before the load that uses it).  Completion is counted by vmcnt like any
// load; the caller waits for it explicitly.  The compiler does not see these
// accesses: it neither waits for them nor moves LDS accesses across them
// ("memory" clobber).
#define MOE_DMA_LINE(V, S) "s_nop 0\n\tbuffer_load_dwordx4 " V ", %[rs], " S " offen lds\n\t"
#define MOE_DMA_NEXT "s_add_u32 m0, m0, 0x400\n\t"

// Four instructions (voff[0..3]).
__device__ __forceinline__ void dma4_rows(i32x4_t rsrc, const uint32_t (&voff)[4], uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %[lds]\n\t"
               MOE_DMA_LINE("%[v0]", "%[so]") MOE_DMA_NEXT MOE_DMA_LINE("%[v1]", "%[so]") MOE_DMA_NEXT
               MOE_DMA_LINE("%[v2]", "%[so]") MOE_DMA_NEXT MOE_DMA_LINE("%[v3]", "%[so]")
               :
               : [v0] "v"(voff[0]), [v1] "v"(voff[1]), [v2] "v"(voff[2]), [v3] "v"(voff[3]),
                 [rs] "s"(rsrc), [so] "s"(__builtin_amdgcn_readfirstlane(soff)),
                 [lds] "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "scc");
}

// Wait until at most N vector-memory instructions of this wave are outstanding
// (they complete in issue order).  vmcnt sits in bits 3:0 and 15:14; expcnt and
// lgkmcnt are left at "no wait".
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70 | 0xf00);
}

__device__ __forceinline__ f32x16 mfma_bf16_32x32x16(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

}  // namespace
}  // namespace moe
