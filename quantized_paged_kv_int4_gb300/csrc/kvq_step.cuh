// Device helpers of the serving-step kernels (plan_step.cu, write_kv.cu, decode_kv.cu).
#pragma once

#include "kvq_device.cuh"

namespace kvq {

constexpr unsigned ERR_FREE = 32u;  // device flag beside those of kvq_device.cuh: a free list ran out

// Start of a kernel that may be launched as a programmatic dependent of the one before it on its stream (any kernel):
// wait until that one has finished and its writes are visible, then let the next launch begin -- in this order, so that
// whatever the next kernel reads ahead of its own wait was finished before this kernel. Every CTA calls it: a grid that
// could end without waiting would release its successor while its predecessor still runs. Back to back, the launch of
// these kernels costs 1 to 3 us less than with plain launches (one-token write 6.1 -> 3.5 us).
// What an earlier kernel may have written is read behind this with plain loads, never through the read-only path (__ldg):
// that one promises that nobody writes the data while the kernel lives, and this kernel lives before its predecessor ends.
__device__ __forceinline__ void pdl_enter() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace kvq
