// ops_args.hpp -- a kernel's arguments, asked for in one go.
#pragma once
#include <hip/hip_runtime.h>

namespace ops {

// Kernel arguments are asked for all at once: read where they are first needed, each
// would be a round trip of its own to memory that no cache near the wave holds.
// (The sizes of the grid and of a workgroup are such arguments too.)
template <class... A>
__device__ __forceinline__ void together(const A&... a)
{
    (([](const A& v) { asm volatile("" ::"s"(v)); })(a), ...);
}

}  // namespace ops
