// One instantiation of the ragged grouped product kernel and its launcher; the
// build compiles this file once per entry of ragged.def with
// -DFP8NT_R_DIR / -DFP8NT_R_SWAP / -DFP8NT_R_PAIR / -DFP8NT_R_BN.
#include <cuda_runtime.h>

#include <atomic>

#include "grouped.h"
#include "kernel_ragged.cuh"

#ifndef FP8NT_R_DIR
#error "FP8NT_R_DIR, FP8NT_R_SWAP, FP8NT_R_PAIR and FP8NT_R_BN must be defined"
#endif

namespace fp8nt {

#define FP8NT_RAGGED_CAT_(d, s, p, n) launch_ragged_d##d##_s##s##_p##p##_bn##n
#define FP8NT_RAGGED_NAME(d, s, p, n) FP8NT_RAGGED_CAT_(d, s, p, n)

cudaError_t FP8NT_RAGGED_NAME(FP8NT_R_DIR, FP8NT_R_SWAP, FP8NT_R_PAIR, FP8NT_R_BN)(const RaggedLaunchArgs &args)
{
    auto kernel = ragged_kernel<FP8NT_R_DIR, FP8NT_R_SWAP != 0, FP8NT_R_PAIR != 0, FP8NT_R_BN>;
    // the shared-memory limit (once per device, the largest possible) and the
    // CTA pairs that can be resident at once
    static std::atomic<int> ready[64];
    if (args.device < 0 || args.device >= 64)
        return cudaErrorInvalidDevice;
    if (ready[args.device].load(std::memory_order_acquire) == 0) {
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, args.max_smem);
        if (err != cudaSuccess)
            return err;
        int n = 1 << 20;
        if (FP8NT_R_PAIR) {
            cudaLaunchConfig_t q = {};
            q.gridDim = dim3(2, 1, 1);
            q.blockDim = dim3(RAGGED_THREADS, 1, 1);
            q.dynamicSmemBytes = (size_t)args.max_smem;
            cudaLaunchAttribute qa[1];
            qa[0].id = cudaLaunchAttributeClusterDimension;
            qa[0].val.clusterDim.x = 2;
            qa[0].val.clusterDim.y = 1;
            qa[0].val.clusterDim.z = 1;
            q.attrs = qa;
            q.numAttrs = 1;
            err = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
            if (err != cudaSuccess)
                return err;
            if (n < 1)
                return cudaErrorInvalidConfiguration;
        }
        ready[args.device].store(n, std::memory_order_release);
    }
    const int pairs = ready[args.device].load(std::memory_order_relaxed);
    int grid = args.grid;
    if (FP8NT_R_PAIR && grid > 2 * pairs)
        grid = 2 * pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(RAGGED_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)args.smem_bytes;
    cfg.stream = args.stream;
    // programmatic dependent launch: set-up may overlap the previous kernel
    // (every thread waits for it before the first global access)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)args.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = args.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, *args.tmap_x, *args.tmap_y, *args.tmap_d, *args.params);
}

} // namespace fp8nt
