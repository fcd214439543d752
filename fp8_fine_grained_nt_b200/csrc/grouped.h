// Host-side interface of the row-grouped operators: what they share with the
// GEMM entry points (device state, tensor maps) and their kernels' launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "ragged_params.h"

namespace fp8nt {

// The current device as the launchers see it (sms: the bound of set_num_sms).
struct DeviceView {
    int index;
    int sms;
    int max_smem;
    unsigned int *status;
    uint64_t timeout_ns;
};
int current_device(DeviceView *out); // a dg_status

// Row-major tensor map of `rank` dimensions (innermost first; `strides` in
// bytes, rank - 1 of them) with the 128-byte swizzle.
int make_tmap_128b(CUtensorMap *map, const void *base, CUtensorMapDataType type, int rank, const uint64_t *dims,
                   const uint64_t *strides, const uint32_t *box);

struct RaggedLaunchArgs {
    const CUtensorMap *tmap_x;
    const CUtensorMap *tmap_y;
    const CUtensorMap *tmap_d;
    const RaggedParams *params;
    int device;
    int max_smem;
    int grid;
    int smem_bytes;
    cudaStream_t stream;
};

typedef cudaError_t (*RaggedLaunchFn)(const RaggedLaunchArgs &);

#define FP8NT_RAGGED(d, s, p, n) cudaError_t launch_ragged_d##d##_s##s##_p##p##_bn##n(const RaggedLaunchArgs &);
#include "ragged.def"
#undef FP8NT_RAGGED

} // namespace fp8nt
