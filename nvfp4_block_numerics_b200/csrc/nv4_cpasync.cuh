// nv4_cpasync.cuh -- asynchronous copies of 4 to 16 bytes into shared memory (cp.async).
#pragma once

#include <cstdint>

namespace nv4 {

// Copies n of kBytes (0 or kBytes) bytes and fills up with zeros.
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, uint32_t n)
{
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}

}  // namespace nv4
