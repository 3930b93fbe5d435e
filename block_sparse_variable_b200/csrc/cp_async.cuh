// cp_async.cuh -- 16-byte asynchronous copies into shared memory.
#pragma once

#include <stdint.h>

namespace bsa {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
  const int n = in ? 16 : 0;  // 0: the 16 bytes are zeros and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

}  // namespace bsa
