// chain.cuh -- kernels of one stream that follow each other closely.  All of
// this library's kernels are launched with programmatic stream serialization:
// a kernel's blocks may start while the kernel before it drains, set up what
// does not depend on it, and wait before they touch global memory.  Every
// kernel waits, so that what came earlier than its predecessor is done too.  A
// block lets the next kernel start once it holds all that it needs of its SM.
#pragma once

#include <cuda_runtime.h>

namespace lapsum {

__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace lapsum
