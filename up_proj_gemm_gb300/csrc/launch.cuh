// Launches that overlap the grid before them on the stream: its last blocks run
// while the next grid is launched and set up (2 us of a back-to-back call). A
// kernel launched so calls grid_wait_previous() in every thread before it
// touches global memory, unless the thread's accesses are ordered behind one
// that did, and grid_launch_next() to let the grid after it do the same. A grid
// that reads something before its wait (a later product of a feed-forward
// call, its weights) relies on the grid before it to have waited first; one that
// needs nothing of the grid before it may wait at its end instead.
// Such a kernel runs while the grid before it still writes, so it reads by plain
// loads: __ldg and restricted pointers are for memory that nobody writes while
// the kernel runs, and a compiler may move them above the wait.
#pragma once
#include <cuda_runtime.h>

#include "mlaq.h"

namespace mlaq {

__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Clusters of `cluster` blocks when that is above 0.
template <typename... Params, typename... Args>
int launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                      cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace mlaq
