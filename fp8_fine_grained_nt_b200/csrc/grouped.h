// Host-side interface of the row-grouped operators: what they share with the
// GEMM entry points (device state, tensor maps) and their kernels' launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "ragged_params.h"

namespace fp8nt {

// The current device as the launchers see it.
struct DeviceView {
    int index;
    int sms;      // the bound of set_num_sms, else all
    bool bounded; // sms is less than the device has
    int max_smem;
    unsigned int *status;
    uint64_t timeout_ns;
};
int current_device(DeviceView *out); // a dg_status

// Clusters of `together` CTAs, one CTA per SM, that run at once on `sms` SMs:
// clusters of 4 and 8 do not fill the GPCs of a 148-SM part (measured: 33, 15).
inline int clusters_held(int together, int sms)
{
    const int most = together == 4 ? 33 : together == 8 ? 15 : 148 / together;
    const int n = sms / together < most ? sms / together : most;
    return n > 0 ? n : 1;
}

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
    int cluster; // CTAs that share a tile
    int smem_bytes;
    cudaStream_t stream;
};

typedef cudaError_t (*RaggedLaunchFn)(const RaggedLaunchArgs &);

#define FP8NT_RAGGED(d, s, p, n) cudaError_t launch_ragged_d##d##_s##s##_p##p##_bn##n(const RaggedLaunchArgs &);
#include "ragged.def"
#undef FP8NT_RAGGED

// Rows grouped by index (csrc/group_rows.cu).  chunk: rows that one CTA takes;
// with more than one chunk, `counts` holds [chunks][groups] ints.  A bound on
// the SMs makes the chunks fewer and longer.
constexpr int GROUP_MAX_CHUNKS = 256;
int group_rows_chunk(int rows, int max_chunks);
cudaError_t launch_group_rows(const void *index, bool i64, int rows, int groups, int alignment, int capacity,
                              int *offsets, int *order, int *slots, int *m_indices, int *counts,
                              const DeviceView &dev, cudaStream_t stream);

// Low-rank adapters: few slots (csrc/lora.cu) and long batches
// (csrc/lora_wide.cu).
constexpr int LORA_MAX_RANK = 256;

struct LoraParams {
    const void *x; // [rows][ld_x]
    const void *lora_a;
    const void *lora_b;
    const float *scales;
    const void *c; // [rows][ld_c]
    void *d;       // [rows][ld_d]
    const int *m_indices;
    const int *order; // null: slot i is row i
    float *v;         // [splits][slots][R]
    unsigned int *status;
    long ld_x, ld_c, ld_d;
    int slots, rows, adapters, R, N, K;
    int k_chunk, splits; // k per CTA of the first kernel, and how many such ranges
    int n_chunk;         // columns per CTA of the second
    int rank_block;      // first block of ranks of a launch of the first kernel
};

long long lora_workspace(int slots, int R, int N, int K); // bytes
cudaError_t launch_lora(const LoraParams &p, bool bf16, const DeviceView &dev, cudaStream_t stream);

// The slots from `first` on, `n` of them, as a call of their own.
inline LoraParams lora_piece(LoraParams p, int first, int n)
{
    p.m_indices += first;
    if (p.order) {
        p.order += first;
    } else { // (slot i is row i; a 16-bit type)
        p.x = static_cast<const char *>(p.x) + 2 * (long)first * p.ld_x;
        p.c = static_cast<const char *>(p.c) + 2 * (long)first * p.ld_c;
        p.d = static_cast<char *>(p.d) + 2 * (long)first * p.ld_d;
        p.rows = p.rows > first ? p.rows - first : 0;
    }
    p.slots = n;
    return p;
}

bool lora_is_wide(int slots, int adapters, int R);
int launch_lora_wide(const LoraParams &p, bool bf16, const DeviceView &dev, cudaStream_t stream); // a dg_status

} // namespace fp8nt
