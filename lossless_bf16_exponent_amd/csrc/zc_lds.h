// Loads straight from memory into LDS and the waits for them, for kernels that
// count their loads themselves (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace zc {
namespace moe {

typedef __attribute__((address_space(3))) void lds_void;

// A wave's loads straight into LDS (16 or 4 bytes a lane, the lanes' results one
// after another from the wave-uniform address in M0), from a uniform base and a
// 32-bit offset a lane.  Inline assembly, so that the compiler adds no waits of
// its own: the kernel counts them.  M0 is an operand, which the compiler sets, so
// that it knows of every change of it.
__device__ __forceinline__ void lds_load16(const uint8_t *base, uint32_t offset, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void lds_load4(const uint8_t *base, uint32_t offset, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(offset), "s"(base), "{m0}"(lds) : "memory");
}
template <int VM>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

}  // namespace moe
}  // namespace zc
