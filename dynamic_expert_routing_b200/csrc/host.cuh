// host.cuh -- host-side helpers shared by the library's translation units: the error message of
// the calling thread, launch tracing (BEAM_TRACE) and the launch of a kernel that belongs to no
// handle.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <utility>

#include "../../include/beam_moe.h"

#define BEAM_HIDDEN __attribute__((visibility("hidden")))

// Records the message returned by beam_moe_last_error and returns `st`.
BEAM_HIDDEN beam_status_t beam_host_fail(beam_status_t st, const char* fmt, ...)
    __attribute__((format(printf, 2, 3)));
BEAM_HIDDEN void beam_host_clear_error();
BEAM_HIDDEN void beam_host_trace(const char* fmt, ...) __attribute__((format(printf, 1, 2)));

// dx [T][d] (rows ld_dx apart) = dlogits [T][C] W^T for W^T given as its rows, w [C][ld_w] (a layer's
// repacked router): beam_router_input_grad with the other order of W.
BEAM_HIDDEN beam_status_t beam_host_input_grad_rows(const float* dlogits, int64_t ld_dlogits, int32_t T, int32_t C,
                                                    const void* w, int32_t w_dtype, int64_t ld_w, int32_t d,
                                                    float* dx, int64_t ld_dx, void* stream);

#define BEAM_HOST_CUDA(call)                                                              \
    do {                                                                                  \
        cudaError_t e_ = (call);                                                          \
        if (e_ != cudaSuccess)                                                            \
            return beam_host_fail(BEAM_ERR_CUDA, "%s failed: %s (%s:%d)", #call,          \
                                  cudaGetErrorString(e_), __FILE__, __LINE__);            \
    } while (0)

// One launch with programmatic stream serialisation: every kernel of the library starts with
// griddepcontrol.wait, so its launch overlaps the tail of the kernel before it.
template <typename... KArgs, typename... Args>
static cudaError_t launch_free(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               cudaStream_t st, Args&&... args)
{
    beam_host_trace("launch grid (%u,%u,%u) block %u smem %zu stream %p", grid.x, grid.y, grid.z,
                    block.x, smem, (void*)st);
    cudaLaunchConfig_t lc = {};
    lc.gridDim = grid;
    lc.blockDim = block;
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kernel, std::forward<Args>(args)...);
    beam_host_trace("  -> %s", cudaGetErrorString(e));
    return e;
}
