// Per-thread asynchronous copies from global into shared memory (cp.async): a
// thread copies ahead what it alone will use, and waits for nothing else.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace zg {

// N (4 or 16) bytes at an N-byte boundary: `bytes` of them from src, the rest 0.
template <int N>
__device__ __forceinline__ void copy_ahead(void* smem, const void* src, int bytes = N)
{
    static_assert(N == 4 || N == 16, "");
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(src), "r"(bytes), "n"(N) : "memory");
}

// Ends the thread's current group of copies / waits until all but its last
// PENDING groups have landed.
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int PENDING>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" :: "n"(PENDING) : "memory");
}

}  // namespace zg
