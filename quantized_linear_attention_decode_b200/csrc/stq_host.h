// stq_host.h -- host-side helpers shared by the files that hold entry points.
#pragma once

#include <cstdlib>
#include <cstring>
#include <type_traits>

#include <nvtx3/nvToolsExt.h>

#include "stq_internal.h"

namespace stq {

inline stq_status cuda_fail(cudaError_t e, const char *what)
{
    return fail_status(e == cudaErrorMemoryAllocation ? STQ_ERR_OOM : STQ_ERR_CUDA, "%s: %s", what,
                       cudaGetErrorString(e));
}

// host-side fault injection: STQ_FAULT names the failure to make
inline bool fault(const char *which)
{
    const char *f = std::getenv("STQ_FAULT");
    return f != nullptr && std::strcmp(f, which) == 0;
}

// STQ_FAULT=timeout: a wait that nothing completes, given a short limit.
inline Waits waits() { return fault("timeout") ? Waits{2000000ull, 16u} : Waits{1000000000ull, 0u}; }

// An NVTX range over a launching call (a no-op unless a profiler is attached),
// so that profiles attribute device work to the entry point that queued it.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// Makes a device current for the duration of a call.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            ok = false;
            return;
        }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
    DeviceGuard(const DeviceGuard &) = delete;
    DeviceGuard &operator=(const DeviceGuard &) = delete;
};

// Bytes of one element of a stq_dtype, 0 if it is none.
inline int dtype_bytes(int32_t dtype) { return dtype == STQ_F32 ? 4 : dtype == STQ_BF16 || dtype == STQ_F16 ? 2 : 0; }

// Launches a kernel whose CTAs may start, and get as far as their wait for the previous grid, while the last CTAs
// of the stream's previous kernel run.  Such a kernel waits in every CTA, so that its end is the end of both.
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, const std::common_type_t<Args> &...args)
{
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
    count_launch();
    return e;
}

// Every head row of `r` starts on a 16-byte boundary.
inline bool rows_aligned(const stq_rows *r, int32_t dtype)
{
    const int64_t per = 16 / dtype_bytes(dtype);
    return reinterpret_cast<uintptr_t>(r->data) % 16 == 0 && r->token_stride % per == 0 && r->head_stride % per == 0;
}

}  // namespace stq
