// Asynchronous copies from global memory into LDS (no VGPR is written), and the
// waits for them.  Lane i's 16 (4) bytes land at m0 + i * 16 (4); m0 is the same
// for every lane.
//
// They are asm strings, since the compiler would wait for all of them before it
// reads LDS.  So it does not see into them either, and the wait states that
// gfx950 asks for stand in the strings: one between the write of m0 and the
// load, and five between a vector instruction's write of a scalar register (the
// readfirstlane that a resource comes from, the reload of a spilled one) and the
// load that reads it, of which the write of m0 is one.  Waiting for both
// everywhere would cost 2.5 % (gate+up of 8192 tokens by 6 of 64 experts, 4096 x
// 7168, bf16: 2.95 and 3.02 ms), so copy16 waits for m0 only: its scalar operands
// are formed long before.  tests/test_lds_copy_waits.py looks for what comes too
// close in the built code.
#pragma once

#include "common.h"

namespace moe {
namespace gemm {

typedef int v4i __attribute__((ext_vector_type(4)));

// Raw buffer resource over `bytes` bytes at p, in scalar registers (gfx9 dword
// 3: 32-bit data, no swizzle; stride 0: what is not at an offset < bytes is not
// read from memory, zeros come in its place).
__device__ __forceinline__ v4i load_rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

#define MOE_M0_WAIT "s_nop 0\n\t"
#define MOE_SGPR_WAIT "s_nop 3\n\t"

// From offset voff + soff of a resource (soff moves the address only, not what
// is checked against its length), 16 or 4 bytes a lane.
__device__ __forceinline__ void copy16(const v4i& r, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %3\n\t" MOE_M0_WAIT "buffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(m0) : "memory", "m0");
}
// To m0 + IMM.
template <int IMM>
__device__ __forceinline__ void copy16(const v4i& r, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_add_u32 m0, %3, %4\n\t" MOE_M0_WAIT "buffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(m0), "n"(IMM) : "memory", "m0", "scc");
}
// Of a resource that has just been formed.
__device__ __forceinline__ void copy16_fresh(const v4i& r, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %3\n\t" MOE_SGPR_WAIT "buffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(m0) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const v4i& r, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %3\n\t" MOE_SGPR_WAIT "buffer_load_dword %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(m0) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const v4i& r, uint32_t voff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\t" MOE_SGPR_WAIT "buffer_load_dword %0, %1, 0 offen lds"
               ::"v"(voff), "s"(r), "s"(m0) : "memory", "m0");
}

// From each lane's own address.
// (lds is made wave-uniform explicitly: inside branches the compiler cannot
// always prove it.)
__device__ __forceinline__ void dma16(const void* g, uint32_t lds) {
  const uint32_t l = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %1\n\t" MOE_M0_WAIT "global_load_lds_dwordx4 %0, off" ::"v"(g), "s"(l)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* g, uint32_t lds) {
  const uint32_t l = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %1\n\t" MOE_M0_WAIT "global_load_lds_dword %0, off" ::"v"(g), "s"(l)
               : "memory", "m0");
}

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_copies() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

}  // namespace gemm
}  // namespace moe
