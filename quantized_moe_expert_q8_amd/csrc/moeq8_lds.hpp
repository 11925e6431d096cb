// LDS building blocks of the staged products: a barrier that leaves global
// loads in flight, and direct global-to-LDS loads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moeq8 {

// Workgroup barrier over LDS only: waits for this wave's LDS operations, not
// for its global loads, so a step's loads stay in flight across it (the
// barrier of __syncthreads also waits for every outstanding global load).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One wave-wide direct load of 16 bytes a lane from global memory into LDS:
// lane i writes LDS bytes [lds + 16 i, lds + 16 i + 16).  `lds` is the
// wave-uniform LDS byte address (the low 32 bits of a shared pointer).  The
// load has no register results; its completion is tracked by vmcnt alone,
// which the caller waits for before any wave reads the bytes (issued this
// way the compiler adds no wait of its own before unrelated LDS reads).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is set here and used by nothing else
__device__ __forceinline__ void load_lds16(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory", "m0");
}
#pragma clang diagnostic pop

// load_lds16 from a wave-uniform base and a byte offset of each lane: no vector
// address arithmetic a load.  The base may come from vector instructions
// (v_readfirstlane), and a vector memory instruction reads an SGPR that such a
// one wrote correctly only 5 wait states later; inside asm nothing inserts
// them.  A scalar move waits by itself, so the load takes its base from one.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16_at(const void* base, uint32_t offset, uint32_t lds) {
    const uint64_t b = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)base >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)base);
    uint64_t at;
    asm volatile("s_mov_b32 m0, %3\n\ts_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0"
                 : "=&s"(at) : "v"(offset), "s"(b), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory", "m0");
}
#pragma clang diagnostic pop

}  // namespace moeq8
