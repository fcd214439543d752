// C-ABI entry points of the row-grouped operators (declared in
// include/fp8_nt.h): argument validation, kernel choice, tensor maps, launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "fp8_nt.h"
#include "grouped.h"

using namespace fp8nt;

namespace {

struct RaggedKernel {
    int dir, swap, pair, bn;
    RaggedLaunchFn launch;
};

const RaggedKernel kRagged[] = {
#define FP8NT_RAGGED(d, s, p, n) {d, s, p, n, launch_ragged_d##d##_s##s##_p##p##_bn##n},
#include "ragged.def"
#undef FP8NT_RAGGED
};
constexpr int kNumRagged = sizeof(kRagged) / sizeof(kRagged[0]);

// test hook: bn, swap << 16, pair << 17 and split << 20 of later calls, 0 = automatic
std::atomic<uint32_t> g_forced_ragged{0};

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

constexpr int kMaxSize = 0x7fff0000; // rows of a product, N and K: 32-bit coordinates, with room for the last tile
constexpr int kMaxSlots = 1 << 30; // rows and slots are counted in 32 bits, with room to round up

// Time of a call in us by a wave model of the tile forms, with the mean rows per
// group (the host does not know more) and counts spread evenly from none to
// twice the mean.  Back to back, these calls run under the power limit (1.2 to
// 1.7 GHz), so the products that a form issues for padding rows cost time even
// where memory bounds the call.  The constants were fitted to calls measured
// that way on B200, every form.  Over 20 calls of NT and NN of 2 to 256 rows per
// group in 1 to 64 groups, the form taken is 2 % slower than the best one on
// average, 13 % at most; where all groups have the same count, which the model
// does not expect, 7 % and 27 % (NN, 8 groups of 128 rows: pairs 57 us, BN = 128
// 45).  TN, 36 calls of 16 to 1024 rows: 1 % and 12 %; same counts 3 % and 24 %.
// Some of them, us, counts spread (SWAP by BN; * the form taken):
//                                           16   32   64  128  128x256  pair
//   NT 16 groups, N=4096, K=7168,  8 rows  139* 145  150  158      151   198
//                                 64 rows  445  240  190  167     169*   241
//                                256 rows            410  324     320*   319
//   NN  8 groups, N=7168, K=2048, 16 rows   58   40*  38   40       56    53
//                                128 rows       109   85   71       64    59*
//   NN 64 groups, N=2112, K=2048, 16 rows  102   90*  85   94       97   126
// and of BN = 16 shared by 1, 2, 4 and 8 CTAs (all groups alike):
//   NT  1 group,  N=256,  K=7168, 10 rows   30   19   13    9*
//   NT 16 groups, N=4096, K=7168,  8 rows  151* 150  145  159
//   NT 64 groups, N=2112, K=2048,  8 rows   89* 100  112  198
//                                          128x128  128x256  pair
//   TN 64 groups, N=2048, K=520, 64 rows       46*       46    51
//                              1024 rows       303      244  211*
//   TN  8 groups, N=7168, K=2048, 16 rows       59      48*    49
double ragged_estimate(const RaggedKernel &k, int split, int groups, int rows, int N, int K, int sms)
{
    const double cycles_per_us = 1900.0;
    const double used = groups < rows ? groups : rows, mean = (double)rows / used;
    const int together = k.pair ? 2 : split;
    const double units = clusters_held(together, sms);
    const int bm = k.pair ? 256 : 128;
    const double stage = 16384.0 + 128.0 * (k.pair ? k.bn / 2 : k.bn);
    if (k.dir == RAGGED_TN || k.dir == RAGGED_TN32) {
        // a tile: its blocks of 64 rows, or its epilogue, whichever is longer
        const double tiles = (double)groups * ceil_div(N, bm) * ceil_div(K, k.bn);
        const double mma = 2.0 * k.bn + 580.0, load = stage / 39.0;
        const double blocks = ceil(mean / 64.0) * (mma > load ? mma : load) + 1100.0;
        const double epilogue = 700.0 + 1450.0 * k.bn / 128.0;
        const double busy = ceil(tiles / units) * (blocks > epilogue ? blocks : epilogue) / cycles_per_us;
        const double memory = ((k.dir == RAGGED_TN32 ? 4.0 : 2.0) * groups * N * K + 2.0 * rows * ((double)N + K)) / 7.0e6;
        return busy > memory ? busy : memory;
    }
    const double out = k.dir == RAGGED_NT ? N : K, red = k.dir == RAGGED_NT ? K : N;
    const double block = k.swap ? k.bn : bm, wide = k.swap ? 128 : k.bn;
    const double tok = 2 * mean <= block ? 1.0 : mean / block + 0.5; // token blocks of a group
    const double tiles = ceil(used * tok * ceil(out / wide));
    const double blocks = ceil(red / 64.0);
    const double mma = (k.swap ? 2.0 * (k.bn < 32 ? 32 : k.bn) : 512.0) + 152.0, load = stage / 61.0;
    // (sharing a tile takes an exchange of about 3000 cycles)
    const double fixed = k.swap ? split > 1 ? 7670.0 : 4670.0 : 7170.0;
    const double tile = (ceil(blocks / split) * (mma > load ? mma : load) + fixed) / cycles_per_us;
    const double weights = 2.0 * wide * red / tok / 8.5e6; // read from memory for one tile
    const double power = 2.0 * tiles * bm * k.bn * blocks * 64.0 / 4.0e9; // all products, padding too
    const double full = floor(tiles / units), rest = tiles - full * units;
    const double wave = tile > units * weights ? tile : units * weights;
    const double last = rest <= 0 ? 0 : tile > rest * weights ? tile : rest * weights;
    // (a shared reduction has to be worth it: 5 %)
    return (full * wave + last + power) * (split > 1 ? 1.05 : 1.0);
}

// The kernel of a call, and the CTAs that share a tile's reduction.
const RaggedKernel *choose_ragged(int dir, int groups, int rows, int N, int K, int sms, int *split)
{
    const uint32_t forced = g_forced_ragged.load(std::memory_order_relaxed);
    const int forced_split = (int)(forced >> 20);
    const long blocks = ceil_div(dir == RAGGED_NT ? K : N, 128); // stages of the swapped tiles
    const RaggedKernel *best = nullptr, *pinned = nullptr;
    double best_us = 0;
    *split = 1;
    for (int i = 0; i < kNumRagged; ++i) {
        const RaggedKernel &k = kRagged[i];
        if (k.dir != dir)
            continue;
        const bool is_pinned =
            ((uint32_t)k.bn | (uint32_t)k.swap << 16 | (uint32_t)k.pair << 17) == (forced & 0xFFFFFu);
        if (k.pair && sms < 2 && !is_pinned) // (a bound on the SMs may leave no room for a pair)
            continue;
        const int most = k.swap && k.bn <= RAGGED_SPLIT_MAX_BN ? RAGGED_MAX_SPLIT : 1;
        for (int s = 1; s <= most && s <= blocks && s <= sms; s *= 2) {
            if (is_pinned) {
                if (!pinned || s == forced_split) {
                    pinned = &k;
                    *split = s;
                }
                continue;
            }
            const double us = ragged_estimate(k, s, groups, rows, N, K, sms);
            if (!pinned && (!best || us < best_us)) {
                best = &k;
                best_us = us;
                *split = s;
            }
        }
    }
    return pinned ? pinned : best;
}

int check_ragged(int dir, const void *A, const void *B, void *D, const int *offsets, int dtype, int G, int M_sum,
                 int N, int K)
{
    if (G <= 0 || M_sum < 0 || N < 0 || K < 0 || (dtype != DG_INPUT_BF16 && dtype != DG_INPUT_F16))
        return DG_ERR_INVALID_ARGUMENT;
    if (G > RAGGED_MAX_GROUPS || N == 0 || K == 0 || N % 8 != 0 || K % 8 != 0)
        return DG_ERR_UNSUPPORTED_SHAPE;
    // bytes of one group's weights: the stride of a tensor map's group axis
    if ((uint64_t)N * (uint64_t)K * 4u >= (1ull << 40))
        return DG_ERR_UNSUPPORTED_SHAPE;
    // the tiles of the smallest tile form are counted in 32 bits
    if (M_sum > kMaxSize || N > kMaxSize || K > kMaxSize ||
        (ceil_div(M_sum, 16) + G) * ceil_div(N > K ? N : K, 128) > 0x7fffffffL ||
        (long)G * ceil_div(N, 128) * ceil_div(K, 128) > 0x7fffffffL)
        return DG_ERR_UNSUPPORTED_SHAPE;
    // without rows only the weight gradient has anything to write
    if (M_sum == 0 && dir != RAGGED_TN)
        return DG_OK;
    if (!D || !offsets || (M_sum > 0 && (!A || !B)))
        return DG_ERR_INVALID_ARGUMENT;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16) || !aligned(offsets, 4))
        return DG_ERR_MISALIGNED;
    return DG_OK;
}

int run_ragged(int dir, const void *A, const void *B, void *D, const int *offsets, int dtype, int d_type,
               int accumulate, int G, int M_sum, int N, int K, cudaStream_t stream)
{
    DeviceView dev;
    int st = current_device(&dev);
    if (st != DG_OK)
        return st;
    const bool tn = dir == RAGGED_TN || dir == RAGGED_TN32;
    if (M_sum == 0) { // the weight gradient of no rows
        if (accumulate)
            return DG_OK;
        const size_t bytes = (size_t)G * N * K * (d_type == RAGGED_OUT_F32 ? 4 : 2);
        return cudaMemsetAsync(D, 0, bytes, stream) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
    }
    int split = 1;
    // (the result's type picks the kernel of a weight gradient)
    const RaggedKernel *k = choose_ragged(dir, G, M_sum, N, K, dev.sms, &split);
    if (!k)
        return DG_ERR_UNSUPPORTED_SHAPE;
    const bool bf16 = dtype == DG_INPUT_BF16;
    const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int bm = k->pair ? 256 : 128;
    const uint32_t y_rows = (uint32_t)(k->pair ? k->bn / 2 : k->bn);

    RaggedParams p;
    memset(&p, 0, sizeof(p));
    p.offsets = offsets;
    p.d = D;
    p.status = dev.status;
    p.timeout_ns = dev.timeout_ns;
    p.num_groups = G;
    p.total_rows = M_sum;
    p.out_type = d_type;
    p.accumulate = accumulate;
    p.split = split;
    const int out = dir == RAGGED_NT ? N : K; // columns of the result
    const int red = dir == RAGGED_NT ? K : N; // reduction of NT, NN
    p.d_rows = N;
    p.d_cols = out;
    const int halves = ragged_halves(k->swap, k->pair);
    p.nkb = (int)ceil_div(red, 64 * halves);
    long tiles;
    if (tn) {
        p.x_blocks = (int)ceil_div(N, bm);
        p.y_blocks = (int)ceil_div(K, k->bn);
        p.tiles_per_group = make_fast_div((uint32_t)p.x_blocks * (uint32_t)p.y_blocks);
        p.last_band = make_fast_div(p.x_blocks % 8 ? (uint32_t)p.x_blocks % 8 : 8u);
        tiles = (long)G * p.x_blocks * p.y_blocks;
    } else {
        p.x_blocks = (int)ceil_div(out, 128);
        p.y_blocks = (int)ceil_div(out, k->bn);
        const long tok_blocks = M_sum / (k->swap ? k->bn : bm) + (G < M_sum ? G : M_sum);
        tiles = tok_blocks * (k->swap ? p.x_blocks : p.y_blocks);
    }
    p.band = make_fast_div(8u * (uint32_t)p.y_blocks);
    const bool x_mn = tn || (dir == RAGGED_NN && k->swap);
    const bool y_mn = tn || (dir == RAGGED_NN && !k->swap);
    p.idesc = ragged_idesc(bf16, x_mn, y_mn, bm, k->bn);

    // shared memory: the deepest operand ring beside the output staging
    const uint32_t stage = (uint32_t)halves * (128u * 128u + y_rows * 128u);
    // (one slot per epilogue warp beside the wide tiles: the stage it leaves room
    // for is worth more, 1728 -> 1491 us for 32768 rows over 8 groups by pairs)
    const int slots = k->swap ? 0 : k->bn == 256 ? 1 : 2;
    int stages = RAGGED_MAX_STAGES;
    for (; stages >= 2; --stages) {
        make_ragged_plan(p, stage, stages, slots, split > 1 ? (uint32_t)k->bn * 512u : 0u);
        if ((int)p.total + 1024 <= dev.max_smem)
            break;
    }
    if (stages < 2)
        return DG_ERR_UNSUPPORTED_SHAPE;

    // operand boxes: 64 reduction elements of all rows (K-major), or 64 rows
    // of the reduction x 64 elements (MN-major); tokens [M_sum][cols], weights
    // [G][N][K]
    auto tokens = [&](CUtensorMap *map, const void *base, int cols, bool mn, uint32_t rows) {
        const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)M_sum}, strides[1] = {(uint64_t)cols * 2};
        const uint32_t box[2] = {64, mn ? 64u : rows};
        return make_tmap_128b(map, base, type, 2, dims, strides, box);
    };
    auto weights = [&](CUtensorMap *map, const void *base, bool mn, uint32_t rows) {
        const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)G};
        const uint64_t strides[2] = {(uint64_t)K * 2, (uint64_t)N * (uint64_t)K * 2};
        const uint32_t box[3] = {64, mn ? 64u : rows, 1};
        return make_tmap_128b(map, base, type, 3, dims, strides, box);
    };
    CUtensorMap tx, ty, td;
    memset(&td, 0, sizeof(td));
    if (tn) {
        st = tokens(&tx, A, N, true, 0);
        if (st == DG_OK)
            st = tokens(&ty, B, K, true, 0);
        if (st == DG_OK) {
            const uint64_t size = d_type == RAGGED_OUT_F32 ? 4 : 2;
            const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)G};
            const uint64_t strides[2] = {(uint64_t)K * size, (uint64_t)N * (uint64_t)K * size};
            const uint32_t box[3] = {(uint32_t)(128 / size), 32, 1};
            st = make_tmap_128b(&td, D, d_type == RAGGED_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                        : d_type == RAGGED_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                3, dims, strides, box);
        }
    } else {
        CUtensorMap *tok = k->swap ? &ty : &tx, *wgt = k->swap ? &tx : &ty;
        st = tokens(tok, A, red, false, k->swap ? y_rows : 128u);
        if (st == DG_OK)
            st = weights(wgt, B, dir == RAGGED_NN, k->swap ? 128u : y_rows);
        if (st == DG_OK && !k->swap) {
            const uint64_t dims[2] = {(uint64_t)out, (uint64_t)M_sum}, strides[1] = {(uint64_t)out * 2};
            const uint32_t box[2] = {64, 32};
            st = make_tmap_128b(&td, D, type, 2, dims, strides, box);
        }
    }
    if (st != DG_OK)
        return st;
    RaggedLaunchArgs args;
    args.tmap_x = &tx;
    args.tmap_y = &ty;
    args.tmap_d = &td;
    args.params = &p;
    args.device = dev.index;
    args.max_smem = dev.max_smem;
    args.cluster = k->pair ? 2 : split;
    const long ctas = tiles * args.cluster;
    const long held = (long)clusters_held(args.cluster, dev.sms) * args.cluster;
    args.grid = (int)(ctas < held ? ctas : held);
    args.smem_bytes = (int)p.total + 1024;
    args.stream = stream;
    return k->launch(args) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

} // namespace

// ====================================================================== C ABI

extern "C" {

int m_grouped_gemm_nt_ragged(const void *A, const void *B, void *D, const int *offsets, int dtype, int num_groups,
                             int M_sum, int N, int K, dg_stream_t stream)
{
    const int st = check_ragged(RAGGED_NT, A, B, D, offsets, dtype, num_groups, M_sum, N, K);
    if (st != DG_OK || M_sum == 0)
        return st;
    return run_ragged(RAGGED_NT, A, B, D, offsets, dtype, dtype, 0, num_groups, M_sum, N, K,
                      reinterpret_cast<cudaStream_t>(stream));
}

int m_grouped_gemm_nn_ragged(const void *A, const void *B, void *D, const int *offsets, int dtype, int num_groups,
                             int M_sum, int N, int K, dg_stream_t stream)
{
    const int st = check_ragged(RAGGED_NN, A, B, D, offsets, dtype, num_groups, M_sum, N, K);
    if (st != DG_OK || M_sum == 0)
        return st;
    return run_ragged(RAGGED_NN, A, B, D, offsets, dtype, dtype, 0, num_groups, M_sum, N, K,
                      reinterpret_cast<cudaStream_t>(stream));
}

int k_grouped_gemm_tn_ragged(const void *A, const void *B, void *D, const int *offsets, int dtype, int d_dtype,
                             int accumulate, int num_groups, int M_sum, int N, int K, dg_stream_t stream)
{
    const int st = check_ragged(RAGGED_TN, A, B, D, offsets, dtype, num_groups, M_sum, N, K);
    if (st != DG_OK)
        return st;
    // the result is FP32 or the operands' type; adding to it needs FP32, so
    // that a sum over many calls is not rounded to 16 bits at each
    if ((d_dtype != DG_INPUT_F32 && d_dtype != dtype) || (accumulate && d_dtype != DG_INPUT_F32))
        return DG_ERR_INVALID_ARGUMENT;
    return run_ragged(d_dtype == DG_INPUT_F32 ? RAGGED_TN32 : RAGGED_TN, A, B, D, offsets, dtype, d_dtype,
                      accumulate != 0, num_groups, M_sum, N, K, reinterpret_cast<cudaStream_t>(stream));
}

int get_row_groups_capacity(int num_rows, int num_groups, int alignment)
{
    if (num_rows < 0 || num_groups <= 0 || alignment <= 0)
        return -DG_ERR_INVALID_ARGUMENT;
    const long most = num_rows < num_groups ? num_rows : num_groups; // groups with rows
    const long cap = (num_rows + most * (long)(alignment - 1) + alignment - 1) / alignment * alignment;
    return cap > kMaxSlots ? -DG_ERR_UNSUPPORTED_SHAPE : (int)cap;
}

long long get_group_rows_workspace_size(int num_rows, int num_groups)
{
    if (num_rows < 0 || num_groups <= 0)
        return -DG_ERR_INVALID_ARGUMENT;
    if (num_groups > RAGGED_MAX_GROUPS || num_rows > kMaxSlots)
        return -DG_ERR_UNSUPPORTED_SHAPE;
    const long chunks = ceil_div(num_rows, group_rows_chunk(num_rows, GROUP_MAX_CHUNKS));
    return chunks > 1 ? (long long)chunks * num_groups * 4 : 0;
}

int group_rows_by_index(const void *index, int index_dtype, int *offsets, int *order, int *slots, int *m_indices,
                        int num_rows, int num_groups, int alignment, void *workspace, size_t workspace_bytes,
                        dg_stream_t stream)
{
    if (index_dtype != DG_INDEX_I32 && index_dtype != DG_INDEX_I64)
        return DG_ERR_INVALID_ARGUMENT;
    const int capacity = get_row_groups_capacity(num_rows, num_groups, alignment);
    if (capacity < 0)
        return -capacity;
    const long long need = get_group_rows_workspace_size(num_rows, num_groups);
    if (need < 0)
        return (int)-need;
    if (!offsets || (num_rows > 0 && (!index || !order)) || (need > 0 && !workspace) ||
        (long long)workspace_bytes < need)
        return DG_ERR_INVALID_ARGUMENT;
    if (!aligned(index, index_dtype == DG_INDEX_I64 ? 8 : 4) || !aligned(offsets, 4) || !aligned(order, 4) ||
        !aligned(slots, 4) || !aligned(m_indices, 4) || !aligned(workspace, 4))
        return DG_ERR_MISALIGNED;
    DeviceView dev;
    const int st = current_device(&dev);
    if (st != DG_OK)
        return st;
    return launch_group_rows(index, index_dtype == DG_INDEX_I64, num_rows, num_groups, alignment, capacity, offsets,
                             order, slots, m_indices, static_cast<int *>(workspace), dev,
                             reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DG_OK
               : DG_ERR_CUDA;
}

long long get_lora_workspace_size(int num_slots, int num_adapters, int rank, int N, int K)
{
    if (num_slots < 0 || num_adapters <= 0 || rank < 0 || N < 0 || K < 0)
        return -DG_ERR_INVALID_ARGUMENT;
    if (num_slots > kMaxSlots || rank == 0 || rank > LORA_MAX_RANK || rank % 8 != 0 || N == 0 || N % 8 != 0 || K == 0 ||
        K % 8 != 0 || N > kMaxSize || K > kMaxSize)
        return -DG_ERR_UNSUPPORTED_SHAPE;
    if (num_slots == 0 || lora_is_wide(num_slots, num_adapters, rank))
        return 0;
    return lora_workspace(num_slots, rank, N, K);
}

int m_grouped_lora_add(const void *x, long long ld_x, const void *lora_a, const void *lora_b, const float *scales,
                       const void *c, long long ld_c, void *d, long long ld_d, const int *m_indices, const int *order,
                       int dtype, int num_slots, int num_rows, int num_adapters, int rank, int N, int K,
                       void *workspace, size_t workspace_bytes, dg_stream_t stream)
{
    if ((dtype != DG_INPUT_BF16 && dtype != DG_INPUT_F16) || num_rows < 0)
        return DG_ERR_INVALID_ARGUMENT;
    const long long need = get_lora_workspace_size(num_slots, num_adapters, rank, N, K);
    if (need < 0)
        return (int)-need;
    if (ld_x < K || ld_c < N || ld_d < N)
        return DG_ERR_INVALID_ARGUMENT;
    if (ld_x % 8 != 0 || ld_c % 8 != 0 || ld_d % 8 != 0)
        return DG_ERR_UNSUPPORTED_SHAPE;
    if (num_slots == 0 || num_rows == 0)
        return DG_OK;
    if (!x || !lora_a || !lora_b || !scales || !c || !d || !m_indices || (need > 0 && !workspace) ||
        (long long)workspace_bytes < need)
        return DG_ERR_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16) || !aligned(c, 16) || !aligned(d, 16) ||
        !aligned(workspace, 16) || !aligned(scales, 4) || !aligned(m_indices, 4) || !aligned(order, 4))
        return DG_ERR_MISALIGNED;
    DeviceView dev;
    const int st = current_device(&dev);
    if (st != DG_OK)
        return st;
    LoraParams p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.lora_a = lora_a;
    p.lora_b = lora_b;
    p.scales = scales;
    p.c = c;
    p.d = d;
    p.m_indices = m_indices;
    p.order = order;
    p.v = static_cast<float *>(workspace);
    p.status = dev.status;
    p.ld_x = (long)ld_x;
    p.ld_c = (long)ld_c;
    p.ld_d = (long)ld_d;
    p.slots = num_slots;
    p.rows = num_rows;
    p.adapters = num_adapters;
    p.R = rank;
    p.N = N;
    p.K = K;
    if (lora_is_wide(num_slots, num_adapters, rank))
        return launch_lora_wide(p, dtype == DG_INPUT_BF16, dev, reinterpret_cast<cudaStream_t>(stream));
    return launch_lora(p, dtype == DG_INPUT_BF16, dev, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DG_OK
               : DG_ERR_CUDA;
}

int dg_force_ragged(int swap_ab, int cta_pair, int block_n, int split)
{
    if (swap_ab == 0 && cta_pair == 0 && block_n == 0 && split == 0) {
        g_forced_ragged.store(0, std::memory_order_relaxed);
        return DG_OK;
    }
    const int most = swap_ab && block_n <= RAGGED_SPLIT_MAX_BN ? RAGGED_MAX_SPLIT : 1;
    if (split < 0 || split > most || (split & (split - 1)) != 0)
        return DG_ERR_UNSUPPORTED_SHAPE;
    for (int i = 0; i < kNumRagged; ++i)
        if (kRagged[i].swap == swap_ab && kRagged[i].pair == cta_pair && kRagged[i].bn == block_n) {
            g_forced_ragged.store((uint32_t)block_n | (uint32_t)swap_ab << 16 | (uint32_t)cta_pair << 17 |
                                      (uint32_t)(split > 0 ? split : 1) << 20,
                                  std::memory_order_relaxed);
            return DG_OK;
        }
    return DG_ERR_UNSUPPORTED_SHAPE;
}

} // extern "C"
