// q8_lds.h -- loads from memory to LDS that go past the registers.  A wave
// waits for its own by count (they complete in order); the compiler does not
// know of them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

__device__ inline uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// 64 lanes x 16 bytes from base + voff to the LDS bytes from `lds` on: kept in
// the caches for others, or read once, past their retention.
#define Q8_LDS_LOAD16(hint) \
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" hint ::"v"(voff), "s"(base), "{m0}"(lds) : "memory");
__device__ inline void lds_load16(uint32_t lds, const uint8_t* base, uint32_t voff) { Q8_LDS_LOAD16("") }
__device__ inline void lds_load16_once(uint32_t lds, const uint8_t* base, uint32_t voff) { Q8_LDS_LOAD16(" nt") }
#undef Q8_LDS_LOAD16

// 64 lanes x 4 bytes.
__device__ inline void lds_load4(uint32_t lds, const uint8_t* base, uint32_t voff) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(voff), "s"(base), "{m0}"(lds)
                 : "memory");
}

// At most N loads (and stores) still on their way.
template <int N>
__device__ inline void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// LDS reads into registers are done: what they read may be overwritten.
__device__ inline void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

}  // namespace q8
