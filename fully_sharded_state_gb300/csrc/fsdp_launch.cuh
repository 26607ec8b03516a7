// fsdp_launch.cuh -- how the operators' kernels follow one another.
//
// An operator is a short chain of kernels on one stream. Each is launched with
// programmatic stream serialisation: its blocks may start, set themselves up
// and wait while the kernel before it still runs. Every kernel launched so
// calls launch_wait() in every block before it touches memory that another
// kernel reads or writes; it returns when all kernels before it have ended
// and what they wrote is visible. launch_next() lets the next kernel start.
#pragma once

#include <cuda_runtime.h>

#include "fsdp_ops_internal.h"

namespace fsdp {
namespace {

__device__ __forceinline__ void launch_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Params, class... Args>
fsdp_status launch(const char *what, void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                   cudaStream_t stream, int cluster, const Args &...args)
{
    if (Record *r = current_record())
        return r->add("%s: %u x %u blocks of %d", what, grid.x, grid.y, threads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    return err == cudaSuccess ? FSDP_OK
                              : set_error(FSDP_ECUDA, "%s launch failed: %s", what, cudaGetErrorString(err));
}

}  // namespace
}  // namespace fsdp
