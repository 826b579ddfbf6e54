// lf_rows.cuh -- what the cache operators' entry points and launches have in
// common: errors, the checks of a tensor of rows, the SM count, and launches as
// programmatic dependents.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/lf.h"

namespace lfr {

inline lf_status status_of(cudaError_t e)
{
    if (e == cudaSuccess) return LF_OK;
    (void)cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? LF_ERR_OUT_OF_MEMORY : LF_ERR_CUDA;
}

inline bool aligned16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows [n][heads][hd]: type, alignment, strides; `written`: no two may overlap.
inline lf_status check_rows(const lf_rows *r, int n, int heads, int hd, bool written)
{
    if (!r) return LF_ERR_INVALID_ARG;
    if (r->dtype != LF_F16 && r->dtype != LF_BF16 && r->dtype != LF_F32) return LF_ERR_NOT_SUPPORTED;
    const long long per16 = r->dtype == LF_F32 ? 4 : 8;   // elements in 16 bytes
    if (!aligned16(r->data) || r->token_stride < 0 || r->head_stride < 0 || r->token_stride % per16 ||
        r->head_stride % per16)
        return LF_ERR_INVALID_ARG;
    const long long most = 1ll << 40;   // elements: keeps every offset far inside 64 bits
    if (r->token_stride > most || r->head_stride > most) return LF_ERR_INVALID_ARG;
    if (written) {
        const long long ts = r->token_stride, hs = r->head_stride;
        const bool t_ok = n == 1 || ts >= hd, h_ok = heads == 1 || hs >= hd;
        const bool apart = n == 1 || heads == 1 || ts >= (heads - 1ll) * hs + hd || hs >= (n - 1ll) * ts + hd;
        if (!t_ok || !h_ok || !apart) return LF_ERR_INVALID_ARG;
    }
    return LF_OK;
}

// Device properties that the plan needs, read once per device.
inline lf_status sm_count(int *out)
{
    static int cached[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return status_of(e);
    if (dev < 64 && cached[dev]) {
        *out = cached[dev];
        return LF_OK;
    }
    e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return status_of(e);
    if (dev < 64) cached[dev] = *out;
    return LF_OK;
}

// Allows a kernel `smem` bytes of dynamic shared memory; ready[device] spares the call once it has been made (the
// attribute is per device, and setting it again is harmless).
template <class F>
inline cudaError_t allow_smem(F *kernel, int smem, bool (&ready)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && ready[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) ready[dev] = true;
    return e;
}

// A launch as a programmatic dependent of the previous kernel on the stream (it waits for that kernel's end before
// any access to global memory), in clusters of `cluster` CTAs along x.
template <class... P, class... A>
inline cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace lfr
