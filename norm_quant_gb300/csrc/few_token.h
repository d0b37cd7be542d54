// few_token.h -- host-side helpers of the few-token operators.  They are kept
// out of common.h, which the combine's kernels are compiled from.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/moe_combine.h"

namespace nqg {

// A launch as a programmatic dependent of the previous kernel on the stream.
struct PdlLaunch {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    PdlLaunch(unsigned grid, unsigned block, size_t smem, moe_stream_t stream)
    {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(block);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = reinterpret_cast<cudaStream_t>(stream);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    PdlLaunch(const PdlLaunch &) = delete;
    template <typename P>
    moe_status run(void (*kern)(P), const P &p) const
    {
        if (cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess)
            return MOE_OK;
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
};

// log2 of an int4 group size (a power of two >= 64), or -1 for any other.
inline int group_shift(int32_t group)
{
    if (group < 64 || (group & (group - 1)) != 0)
        return -1;
    int s = 6;
    while ((1 << s) < group)
        ++s;
    return s;
}

} // namespace nqg
