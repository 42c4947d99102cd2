// context.h — the current device as the entry points outside moe_api.cu need it.
#pragma once

#include "internal.h"

namespace moe {

struct DeviceContext {
    int num_sms;
    WaitCfg wait;  // the limit of moe_set_wait_limit_ns and the library's device error word
};

// Fills `out` for the current device; a moe_status_t.
int device_context(DeviceContext &out);

// 16-bit floating-point tensor map of a stack [n, rows, cols] with a row pitch and a matrix
// pitch in elements (boxes of box_cols columns x box_rows rows of one matrix, 64 columns with
// 128-byte swizzle or 32 with 64-byte swizzle; elements outside a matrix read as zero). False if the driver rejects it.
bool map_stack_f16(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t n, int64_t pitch,
                   int64_t mat_pitch, uint32_t box_cols, uint32_t box_rows);

// Programmatic dependent launch. A kernel launched with launch_dependent may start while the one
// before it in the stream still runs, from the moment all of that one's blocks have called
// allow_dependents; dependency_wait returns once the one before has finished and its writes are
// visible. What was enqueued before that one has finished already if that one was launched
// normally or has itself waited before it allowed dependents.
__device__ __forceinline__ void dependency_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void allow_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <class Kernel, class... Args>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                             Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe
