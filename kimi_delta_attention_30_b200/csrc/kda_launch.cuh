// Kernels of one call that follow one another closely: the later one may be brought onto the
// machine while the earlier one still runs, forms what it can from the call's inputs and then
// waits for the earlier one's results.  The gap between two dependent launches, 1 to 2 us, and
// the later kernel's start go from the path that way.
//
// The first kernel of a call is launched the ordinary way, so the call's inputs are complete
// before any kernel launched here begins.  Every block of such a kernel waits before it ends or
// writes.  What the earlier kernels wrote is read behind the wait through pointers that are not
// __restrict__, or with __ldcg or bulk copies: a load that takes the data for constant could
// move ahead of it.  So too the tables of sequences, where their kernel is the one before; a
// kernel that reads them as constants, and the first behind them then, has an ordinary launch.
#pragma once

#include <cuda_runtime.h>

namespace kda {

// Results of the kernels before are complete and visible behind this.
__device__ __forceinline__ void wait_for_kernels_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Once every block has come here (or ended), the next kernel's blocks may start.
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A&&... args) {
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = early;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kern, P(args)...);
    if (e != cudaSuccess) cudaGetLastError();   // reported by the call, and not once more by the next one
    return e;
}

}  // namespace kda
