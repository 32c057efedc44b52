// cbq_copy.cuh -- copies to shared memory that a thread does not wait for.
#pragma once

#include <stdint.h>

namespace cbq {

// 16 bytes to shared memory, or 16 zero bytes where put is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool put) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(put ? 16 : 0) : "memory");
}
// The same for 4 bytes.
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool put) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(put ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace cbq
