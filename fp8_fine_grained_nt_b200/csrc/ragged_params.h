// Parameters and shared-memory plan of the ragged grouped products
// (kernel_ragged.cuh), shared by the host launcher and the kernel.
#pragma once

#include <stdint.h>

#include "params.h"

namespace fp8nt {

enum RaggedDir : int { RAGGED_NT = 0, RAGGED_NN = 1, RAGGED_TN = 2, RAGGED_TN32 = 3 }; // TN32: FP32 result
enum RaggedOut : int { RAGGED_OUT_F32 = 0, RAGGED_OUT_BF16 = 1, RAGGED_OUT_F16 = 2 };

// 64-wide blocks of the reduction (128-byte swizzled rows) per stage.  Two where
// three such stages fit: the thread that issues the MMAs then waits and commits
// half as often, and it is what holds these kernels back (N = 4096, K = 7168, pairs:
// 1590 -> 1491 us back to back for 32768 rows over 8 groups; swapped: 157 -> 152 us
// for 128 rows over 16).
__host__ __device__ constexpr int ragged_halves(bool swap, bool pair)
{
    return pair || swap ? 2 : 1;
}
constexpr int RAGGED_THREADS = 384;     // 12 warps, 8 of them in the epilogue
constexpr int RAGGED_PARTIAL = 512;     // TN32: rows per partial sum
constexpr int RAGGED_REGS_OTHER = 56;   // TN32: registers of warps 0-3 and of the epilogue warps
constexpr int RAGGED_REGS_EPILOGUE = 224;
static_assert(4 * 32 * RAGGED_REGS_OTHER + 8 * 32 * RAGGED_REGS_EPILOGUE <= RAGGED_THREADS * REGS_AT_LAUNCH,
              "register split exceeds the launch allocation");
constexpr int RAGGED_SPLIT_MAX_BN = 64;  // swapped tiles that the CTAs of a cluster may share
constexpr int RAGGED_MAX_SPLIT = 8;
constexpr int RAGGED_MAX_STAGES = 12;
constexpr int RAGGED_MAX_GROUPS = 1024;
constexpr uint32_t RAGGED_SLOT_BYTES = 4096; // output staging: 32 rows of 128 bytes

// Unsigned division by a constant for n < 2^31: q = (umulhi(n, mul) + n) >> shift
// (Granlund and Montgomery's method).
struct FastDiv {
    uint32_t d, mul, shift;
};

inline FastDiv make_fast_div(uint32_t d)
{
    FastDiv f;
    f.d = d;
    f.shift = 0;
    while ((1ull << f.shift) < d)
        ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
    return f;
}

struct RaggedParams {
    const int *offsets; // [num_groups + 1] segment bounds
    void *d;
    unsigned int *status;
    uint64_t timeout_ns;
    int num_groups;
    int total_rows;      // rows of the token tensors
    int d_rows;          // TN: rows of one group's result (N)
    int d_cols;          // columns of the result
    int nkb;             // NT, NN: blocks (64 * ragged_halves wide) of the reduction
    int x_blocks;        // SWAP: blocks of 128 output columns; TN: blocks of X rows
    int y_blocks;        // NT, NN without SWAP: blocks of output columns; TN: blocks of Y rows
    FastDiv tiles_per_group; // TN
    FastDiv band;        // without SWAP: tiles of 8 X blocks; with it: token blocks take the slow way
    FastDiv last_band;   // TN: X blocks of the last band
    int out_type;        // RaggedOut
    int accumulate;      // TN32: add to the result
    uint32_t idesc;      // tcgen05.mma instruction descriptor
    int split;           // SWAP: CTAs (a cluster) that share a tile's reduction; 1, 2, 4 or 8
    int stages;
    int out_slots;       // staging slots per epilogue warp (0 with SWAP)
    uint32_t off_out;
    uint32_t off_recv;   // split: the sums received, BN token rows of 128 FP32 columns
    uint32_t off_groups; // tile prefix [G + 1], first row [G], rows [G]
    uint32_t off_bars;
    uint32_t off_misc;   // tensor-memory address, abort flag, scan partials
    uint32_t total;      // bytes, excluding the 1024-byte alignment slack
};

// Operand ring of `stages`, staging, received sums, group table, barriers.
inline void make_ragged_plan(RaggedParams &p, uint32_t stage_bytes, int stages, int out_slots, uint32_t recv_bytes)
{
    p.stages = stages;
    p.out_slots = out_slots;
    p.off_out = stage_bytes * (uint32_t)stages;
    p.off_recv = p.off_out + 8u * (uint32_t)out_slots * RAGGED_SLOT_BYTES;
    p.off_groups = p.off_recv + recv_bytes;
    p.off_bars = align_up_u32(p.off_groups + 4u * (3u * (uint32_t)p.num_groups + 1u), 8);
    p.off_misc = align_up_u32(p.off_bars + 8u * (4u * RAGGED_MAX_STAGES + 8u), 16);
    p.total = p.off_misc + 80;
}

// tcgen05.mma kind::f16: FP32 result, both operands BF16 (or FP16), `mn` set
// where the operand's i / j index is the contiguous one, M x N per MMA.
inline uint32_t ragged_idesc(bool bf16, bool x_mn, bool y_mn, int m, int n)
{
    const uint32_t type = bf16 ? 1u : 0u;
    return (1u << 4) | (type << 7) | (type << 10) | ((x_mn ? 1u : 0u) << 15) | ((y_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

} // namespace fp8nt
