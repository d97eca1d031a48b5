// hkv_host.h -- host-side state and checks shared by the library's sources.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "hkv.h"

namespace hkv {

// Defined in hkv_api.cu.
extern std::atomic<uint64_t> g_launches;  // kernels launched by this process
extern std::atomic<uint64_t> g_wait_ns;   // bound of every spin-wait
extern std::atomic<int32_t> g_withhold;   // hkv_debug_withhold_publish

int es_of(hkv_dtype d);
int sm_count();  // of the current device; 0 when it cannot be queried
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
hkv_status check_problem(const hkv_problem *p);
hkv_status check_tier(const hkv_tier *t, const hkv_problem *p, bool need_v);
// Per-device kernel attributes (dynamic shared memory opt-in, resident CTAs per SM).
hkv_status prepare(const void *fn, int threads, size_t smem, int *blocks_per_sm);

inline bool ptr_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Bytes that a call reads or writes.
struct Span {
    const void *p;
    int64_t bytes;
    bool meets(const Span &x) const
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(x.p);
        return a < b ? b - a < (uintptr_t)bytes : a - b < (uintptr_t)x.bytes;
    }
};

// Launch `kernel` as a programmatic dependent of the previous kernel on the
// stream (it calls wait_prior_grid() before it reads that kernel's results);
// cluster: CTAs per cluster (1 = none).
template <typename P>
hkv_status launch_dependent(void (*kernel)(P), int64_t grid, int threads, size_t smem, cudaStream_t stream,
                            const P &params, int cluster = 1)
{
    if (grid <= 0)
        return HKV_OK;
    const hkv_status s = prepare(reinterpret_cast<const void *>(kernel), threads, smem, nullptr);
    if (s != HKV_OK)
        return s;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess)
        return HKV_ERR_CUDA;
    g_launches.fetch_add(1);
    return HKV_OK;
}

}  // namespace hkv
