// Launches with attributes: clusters, and kernels that may overlap the one
// before them.
#pragma once

#include "sg_internal.cuh"

// `after`: the kernel before it in the stream is one of this call's, which this
// one may overlap.  It waits for that one's end (grid_wait) before it uses anything
// that the call writes, and before it ends, so that the next kernel's wait reaches
// all of them.  A call's first kernel is launched without: nothing says that a
// kernel of the program's before it waited in its turn, and the wait does not reach
// past that one.
template <typename... P, typename... A>
sg_status launch(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, bool after, cudaStream_t st,
                 A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    cfg.attrs = at;
    cfg.numAttrs = 0;
    if (cluster > 1) {
        at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
        at[cfg.numAttrs].val.clusterDim.y = 1;
        at[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    if (after) {
        at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    SG_TRY_CUDA(cudaLaunchKernelEx(&cfg, kernel, args...));
    return SG_OK;
}
