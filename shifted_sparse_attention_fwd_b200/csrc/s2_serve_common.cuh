// Pieces shared by the serving kernels (append, decode, prompt): their ids in the device error
// word, the paged cache's addresses, and programmatic dependent launch.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace s2 {

// Ids beside those of s2_device.cuh; code = (kernel id << 8) | site. Sites of the second kind are
// no waits: an index that the caller's arrays hold lies outside the cache.
enum ServeKernelId : uint32_t { KID_APPEND = 6, KID_DECODE = 7, KID_PROMPT = 8 };
constexpr uint32_t kSiteBadIndex = 0x80;   // sites from here on are bad indices
constexpr uint32_t kSiteBadPage = 0x80;    // a page number outside [0, pages)
constexpr uint32_t kSiteBadLength = 0x81;  // a length outside the block table's row

// One half (K or V) of a paged cache: element (page, slot, h, c) at p + page * sp + slot * st +
// h * d + c. Offsets are 64-bit: a cache passes 2^31 elements at 4096 pages of 64 tokens x 64
// heads x 128.
struct PagedRef {
  __nv_bfloat16* p;
  long long sp, st;
};

__device__ __forceinline__ void report_bad_index(unsigned int* err, uint32_t kernel, uint32_t site) {
  atomicCAS(err, 0u, (kernel << 8) | site);
}

// Programmatic dependent launch. The serving kernels are launched so that they may start before the
// kernel in front of them in the stream has ended: they wait for it (its whole grid, with its memory
// operations) before they touch any memory of the caller's, and let the kernel behind them, if it is
// launched the same way, start as early. A step's kernels take 3 to 6 us each, of which a launch is 1.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace s2
