// Persistent tcgen05 kernel for 16-bit (BF16 or FP16) matrix products grouped
// by expert over row segments of any length, in the three directions of a
// grouped linear layer.  Segment g is rows [offsets[g], offsets[g + 1]).
//
//   NT (forward)          d[t, n]    = sum_k a[t, k] b[g, n, k]
//   NN (input gradient)   d[t, k]    = sum_n a[t, n] b[g, n, k]
//   TN (weight gradient)  d[g, n, k] = sum_{t in g} a[t, n] b[t, k]
//
// All three are P[i, j] = sum_r X[i, r] Y[j, r] over 64-wide blocks of r, and
// the tensor core reads an operand either with r contiguous ("K-major") or
// with i / j contiguous ("MN-major"), so no operand is ever transposed in
// memory: NT reads both K-major, NN reads b MN-major, TN reads both MN-major.
// Accumulation is FP32 in tensor memory over the whole reduction; the result
// is rounded once, on store.  The tensor core rounds each step of 16 towards
// zero, a bias that grows with the length: nothing beside the rounding to 16
// bits, but 4e-6 of an FP32 weight gradient over 2048 rows (and 3e-5 over
// 16384).  So FP32 results (direction TN32) are added up in registers, rounded
// to nearest, from partial sums of 512 rows: 5e-7, for 4 % of the time (452 ->
// 469 us back to back at 16384 rows of 8 groups, N = 7168, K = 2048).
//
// Tile forms:
//   PAIR   256 x 256 by a cluster of two CTAs (cta_group::2): each CTA loads
//          its own 128 rows of X and half of Y, so per CTA a 64-wide block
//          brings 32 KB for 512 cycles of MMA.  For many rows per group and
//          for weight gradients.
//   single 128 x BN by one CTA.
//   SWAP   the weights are X (128 of the output's columns per tile) and BN
//          token rows are Y: for few rows per group, where the call is bound
//          by reading the weights and 128 token rows would be mostly padding.
//          Where there are too few such tiles to fill the SMs, the CTAs of a
//          cluster share one: each sums a range of the reduction, sends every
//          other CTA the part of its FP32 sums that the other one owns (token
//          rows) through distributed shared memory, and adds up what it
//          receives in rank order.
//
// Long groups are bound by the tensor core: 8192 x 8192 x 8192 takes 686 us
// alone, 1603 TFLOP/s (a library product of that size: 650 us); back to back,
// under the power limit, 812 us (776).  Few rows per group are bound by reading
// the weights: 128 rows over 16 groups, N = 4096, K = 7168, 152 us, 6.2 TB/s.
// Weight gradients of short groups are bound by writing the result as far as
// its rows are whole 32-byte sectors and its columns fill the tiles: 1999 rows
// over 64 groups, 2048 x 512 into BF16, 33 us for 134 MB (a plain fill of them
// takes 36).  528 columns take 39 us, for a fifth tile of 128, as do 576 (640: 40);
// 520 take 44: every other boundary between rows lies within a sector.
// Tiles go to the CTAs in turn, whatever their groups' lengths: in the case of
// 16384 rows above the busiest pair has 8 % more rows than the mean.
//
// Roles (384 threads, one CTA per SM): warp 0 TMA producer, warp 1 TMEM
// allocator and MMA issuer, warp 2 clears the rows behind a segment's end (TN
// only), warp 3 hands back received sums (shared reductions), warps 4-11
// epilogue (a 32-lane quarter of tensor memory and half of the tile's columns
// each).  Two accumulators in tensor memory let a tile's epilogue overlap the
// next tile's MMAs.
#pragma once

#include "kernel.cuh"
#include "ragged_params.h"

namespace fp8nt {

template <int DIR, bool SWAP, bool PAIR, int BN>
struct RaggedTraits {
    static_assert(!PAIR || (BN == 256 && !SWAP), "a CTA pair computes 256 x 256");
    static constexpr bool TN = DIR == RAGGED_TN || DIR == RAGGED_TN32;
    static_assert(!TN || !SWAP, "the weight gradient has no swapped form");
    static constexpr int BM = PAIR ? 256 : 128;      // rows of X per tile
    static constexpr int Y_ROWS = PAIR ? BN / 2 : BN; // rows of Y each CTA loads
    // a side is MN-major where its i / j index is the contiguous one in memory
    static constexpr bool X_MN = TN || (DIR == RAGGED_NN && SWAP);
    static constexpr bool Y_MN = TN || (DIR == RAGGED_NN && !SWAP);
    static_assert(!Y_MN || Y_ROWS % 64 == 0, "MN-major operands load in 64-wide chunks");
    static constexpr uint32_t X_BYTES = 128 * 128; // 64 of the reduction
    static constexpr uint32_t Y_BYTES = Y_ROWS * 128;
    static constexpr uint32_t HALF_BYTES = X_BYTES + Y_BYTES;
    // 64-wide blocks of the reduction per stage: with two, one wait and one
    // commit serve eight MMAs
    static constexpr int H = ragged_halves(SWAP, PAIR);
    static constexpr int BK = 64 * H;
    static constexpr uint32_t STAGE_BYTES = H * HALF_BYTES;
    static constexpr int TMEM_COLS = 2 * BN;
    static_assert((TMEM_COLS & (TMEM_COLS - 1)) == 0 && TMEM_COLS <= 512, "power of two, at most 512");
};

struct RaggedTile {
    int g;
    int first; // first row of the group's segment
    int rows;  // rows of the segment
    int i0;    // tile's first X row: token (relative to the segment) or output index
    int j0;    // tile's first Y row
    int nkb;   // blocks (stages, BK wide) of the reduction
};

__device__ __forceinline__ int fast_div(int n, const FastDiv &f)
{
    return (int)((__umulhi((uint32_t)n, f.mul) + (uint32_t)n) >> f.shift);
}

// Tile t.  `tiles` holds the tile prefix sums of the groups (NT, NN); `g` is
// the group of the caller's previous (lower) tile.  Order within a group: bands
// of 8 X blocks, X fastest within a band, so that the tiles in flight share
// both operands in L2 (8192 x 8192 x 8192: bands of 4 and of 16 were 2 % slower).
// SWAP: the token blocks of one weight block run side by side.
template <int DIR, bool SWAP, int BM, int BN, int BK>
__device__ __forceinline__ RaggedTile ragged_tile(const RaggedParams &p, int t, int &g, const int *tiles,
                                                  const int *first, const int *count)
{
    constexpr bool TN = DIR == RAGGED_TN || DIR == RAGGED_TN32;
    RaggedTile r;
    int local, xb, yb;
    if (TN) {
        g = fast_div(t, p.tiles_per_group);
        local = t - g * (int)p.tiles_per_group.d;
        xb = p.x_blocks;
        yb = p.y_blocks;
    } else {
        if (t >= tiles[g + 1]) {
            int lo = g + 1, hi = p.num_groups - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tiles[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            g = lo;
        }
        local = t - tiles[g];
        const int tok_blocks = (count[g] + (SWAP ? BN : BM) - 1) / (SWAP ? BN : BM);
        xb = SWAP ? p.x_blocks : tok_blocks;
        yb = SWAP ? tok_blocks : p.y_blocks;
    }
    r.g = g;
    r.first = first[g];
    r.rows = count[g];
    if (SWAP) {
        const int q = yb == 1 ? local : local / yb;
        r.i0 = q * BM;
        r.j0 = (local - q * yb) * BN;
    } else {
        const int band = fast_div(local, p.band);
        const int in_band = local - band * (int)p.band.d;
        const int width = xb - band * 8;
        int y;
        if (width >= 8)
            y = in_band >> 3;
        else if (TN)
            y = fast_div(in_band, p.last_band);
        else
            y = in_band / width;
        r.i0 = (band * 8 + in_band - y * min(width, 8)) * BM;
        r.j0 = y * BN;
    }
    r.nkb = TN ? (r.rows + BK - 1) / BK : p.nkb;
    return r;
}

__device__ __forceinline__ bool wait_ragged(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_flag,
                                            const RaggedParams &p)
{
    const uint32_t a = smem_addr(bar);
    return mbar_try_wait(a, parity) || wait_slow(a, parity, abort_flag, p.status, p.timeout_ns, true);
}

__device__ __forceinline__ void drain_ragged(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_flag,
                                             const RaggedParams &p)
{
    const uint32_t a = smem_addr(bar);
    if (!mbar_try_wait(a, parity))
        wait_slow(a, parity, abort_flag, p.status, p.timeout_ns, false);
}

// The same for a barrier that other CTAs of the cluster arrive on after writing
// this one's shared memory, or after reading what this one is to write again.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_flag,
                                             const RaggedParams &p)
{
    // (a fence would also wait for this thread's own stores on their way)
    const bool got = wait_ragged(bar, parity, abort_flag, p);
    mbar_acquire_cluster(smem_addr(bar), parity);
    return got;
}

// One operand's 64-wide reduction block: K-major, one box of ROWS rows of 128
// bytes; MN-major, ROWS / 64 boxes of 64 reduction rows of 128 bytes.
// GROUPED: the tensor has a group axis.  LEADER: completion is counted on the
// pair leader's barrier at cluster address `bar`.
template <bool MN, bool GROUPED, bool LEADER, int ROWS>
__device__ __forceinline__ void ragged_load(uint8_t *dst, const CUtensorMap *map, uint32_t bar, int mn, int red, int g)
{
#pragma unroll
    for (int c = 0; c < (MN ? ROWS / 64 : 1); ++c) {
        const int x = MN ? mn + 64 * c : red;
        const int y = MN ? red : mn;
        tma_load_nd<GROUPED, LEADER>(dst + c * 8192, map, bar, x, y, g);
    }
}

// Shared-memory descriptor of an operand at `saddr`: K-major as make_sdesc;
// MN-major, 64 elements (128 bytes, swizzled) along i / j, 8-row groups of the
// reduction 1024 bytes apart, the next 64 elements 8192 bytes on.
template <bool MN>
__device__ __forceinline__ uint64_t ragged_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(MN ? 8192u >> 4 : 1u) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// Two FP32 values rounded to nearest even in the result's 16-bit type.
__device__ __forceinline__ uint32_t pack_16x2(float lo, float hi, bool bf16)
{
    if (bf16)
        return pack_bf16x2(lo, hi);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DIR, bool SWAP, bool PAIR, int BN>
__global__ void __launch_bounds__(RAGGED_THREADS, 1)
    ragged_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_y,
                  const __grid_constant__ CUtensorMap tmap_d, const __grid_constant__ RaggedParams p)
{
    using T = RaggedTraits<DIR, SWAP, PAIR, BN>;
    constexpr bool TN = T::TN;
    constexpr bool F32 = DIR == RAGGED_TN32;
    constexpr int PARTIAL = RAGGED_PARTIAL / T::BK; // stages per partial sum
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stages = (uint32_t)p.stages;

    uint64_t *full = reinterpret_cast<uint64_t *>(smem + p.off_bars); // stage holds its operands
    uint64_t *empty = full + RAGGED_MAX_STAGES;                       // its MMAs have completed
    uint64_t *tail_full = empty + RAGGED_MAX_STAGES;                  // TN: a segment's last block landed here
    uint64_t *tail_ready = tail_full + RAGGED_MAX_STAGES;             // and its foreign rows are cleared
    uint64_t *acc_full = tail_ready + RAGGED_MAX_STAGES;              // accumulator complete (x2)
    uint64_t *acc_empty = acc_full + 2;                               // accumulator read (x2)
    uint64_t *mma_done = acc_empty + 2;
    uint64_t *recv_full = mma_done + 1; // split: every CTA's sums for this one's token rows are here
    uint64_t *recv_free = recv_full + 1; // split: every CTA has read what this one sent
    uint64_t *recv_read = recv_free + 1; // split: this CTA's epilogue has read what it received
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + p.off_misc);
    volatile uint32_t *abort_flag = misc + 1;
    int *tiles = reinterpret_cast<int *>(smem + p.off_groups);
    int *first = tiles + p.num_groups + 1;
    int *count = first + p.num_groups;

    // ---------------------------------------------------------------- set-up
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&tail_full[s], 1);
            mbar_init(&tail_ready[s], PAIR ? 2 : 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], PAIR ? 16 : 8);
        }
        mbar_init(mma_done, 1);
        mbar_init(recv_full, 4u * (uint32_t)p.split);
        mbar_init(recv_free, (uint32_t)p.split);
        mbar_init(recv_read, 8);
        misc[1] = 0u;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmap_x);
        tma_prefetch_desc(&tmap_y);
        tma_prefetch_desc(&tmap_d);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(misc, T::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(misc, T::TMEM_COLS);
            tmem_relinquish();
        }
    }
    // the previous kernel's results are visible from here on; a next one may
    // set itself up
    grid_dependency_wait();
    grid_launch_dependents();
    // Segments.  Each thread takes `per` consecutive groups; exclusive prefix
    // sums of their tiles by a block scan.  A bad offset is flagged, and then
    // one thread clamps every segment into the rows behind the one before it:
    // segments that overlap would have more tiles than can be counted.
    {
        const int per = (p.num_groups + RAGGED_THREADS - 1) / RAGGED_THREADS;
        const int g0 = threadIdx.x * per;
        int mine = 0;
        int bad = 0;
        for (int g = g0; g < min(g0 + per, p.num_groups); ++g) {
            const int lo = __ldg(p.offsets + g), hi = __ldg(p.offsets + g + 1);
            const int a = min(max(lo, 0), p.total_rows);
            const int b = min(max(hi, a), p.total_rows);
            bad |= lo != a || hi != b;
            first[g] = a;
            count[g] = b - a;
        }
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0) {
                atomicOr(p.status, DEVERR_BAD_INDEX);
                for (int g = 0, at = 0; g < p.num_groups; ++g) {
                    first[g] = min(max(__ldg(p.offsets + g), at), p.total_rows);
                    at = min(max(__ldg(p.offsets + g + 1), first[g]), p.total_rows);
                    count[g] = at - first[g];
                }
            }
            __syncthreads();
        }
        if (!TN) {
            for (int g = g0; g < min(g0 + per, p.num_groups); ++g) {
                constexpr int TOK = SWAP ? BN : T::BM;
                mine += (count[g] + TOK - 1) / TOK * (SWAP ? p.x_blocks : p.y_blocks);
            }
            int incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d)
                    incl += v;
            }
            if (lane == 31)
                misc[4 + warp] = (uint32_t)incl;
            __syncthreads();
            int at = incl - mine;
            for (int w = 0; w < warp; ++w)
                at += (int)misc[4 + w];
            for (int g = g0; g < min(g0 + per, p.num_groups); ++g) {
                constexpr int TOK = SWAP ? BN : T::BM;
                tiles[g] = at;
                at += (count[g] + TOK - 1) / TOK * (SWAP ? p.x_blocks : p.y_blocks);
            }
            if (threadIdx.x == RAGGED_THREADS - 1)
                tiles[p.num_groups] = at;
        }
    }
    tc_fence_before();
    const bool split = SWAP && p.split > 1;
    if (PAIR || split)
        cluster_sync(); // the others may arrive on this CTA's barriers from here on
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = misc[0];
    const int num_tiles = TN ? p.num_groups * (int)p.tiles_per_group.d : tiles[p.num_groups];
    const uint32_t rank = PAIR || split ? cluster_ctarank() : 0u;
    const bool leader = !PAIR || rank == 0; // issues the MMAs
    const int per_tile = PAIR ? 2 : SWAP ? p.split : 1; // CTAs that share a tile
    const int t_first = (int)blockIdx.x / per_tile;
    const int t_stride = (int)gridDim.x / per_tile;
    // split: this CTA's range of the reduction
    const int kb_first = SWAP ? (int)((long)p.nkb * rank / p.split) : 0;
    const int kb_count = SWAP ? (int)((long)p.nkb * (rank + 1) / p.split) - kb_first : 0;
    int group = 0; // of the role's current tile

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if constexpr (F32)
            regs_dec<RAGGED_REGS_OTHER>();
        if (lane == 0) {
            uint32_t it = 0, s = 0, phase = 1;
            // per stage: its last use was counted on full[], and the parity of
            // its uses of full[]
            uint32_t plain = 0, uses = 0;
            bool ok = true;
            for (int t = t_first; ok && t < num_tiles; t += t_stride) {
                const RaggedTile ti = ragged_tile<DIR, SWAP, T::BM, BN, T::BK>(p, t, group, tiles, first, count);
                const int x_mn = ti.i0 + (PAIR ? (int)rank * 128 : 0) + ((!TN && !SWAP) ? ti.first : 0);
                const int y_mn = ti.j0 + (PAIR ? (int)rank * T::Y_ROWS : 0) + (SWAP ? ti.first : 0);
                const int red0 = TN ? ti.first : kb_first * T::BK;
                const int nkb = SWAP ? kb_count : ti.nkb;
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!wait_ragged(&empty[s], phase, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = smem + s * T::STAGE_BYTES;
                    const int red = red0 + kb * T::BK;
                    const bool tail = TN && ti.rows - kb * T::BK < T::BK;
                    if (tail) {
                        // counted by each CTA for itself: warp 2 clears the
                        // rows of other segments before the MMAs read them
                        mbar_arrive_expect_tx(&tail_full[s], T::STAGE_BYTES);
                        const uint32_t bar = smem_addr(&tail_full[s]);
#pragma unroll
                        for (int h = 0; h < T::H; ++h, dst += T::HALF_BYTES) {
                            ragged_load<T::X_MN, false, false, 128>(dst, &tmap_x, bar, x_mn, red + 64 * h, ti.g);
                            ragged_load<T::Y_MN, false, false, T::Y_ROWS>(dst + T::X_BYTES, &tmap_y, bar, y_mn,
                                                                          red + 64 * h, ti.g);
                        }
                        plain &= ~(1u << s);
                    } else {
                        if (leader)
                            mbar_arrive_expect_tx(&full[s], PAIR ? 2 * T::STAGE_BYTES : T::STAGE_BYTES);
                        const uint32_t bar =
                            PAIR ? map_shared_rank(smem_addr(&full[s]), 0u) : smem_addr(&full[s]);
#pragma unroll
                        for (int h = 0; h < T::H; ++h, dst += T::HALF_BYTES) {
                            ragged_load<T::X_MN, SWAP, PAIR, 128>(dst, &tmap_x, bar, x_mn, red + 64 * h, ti.g);
                            ragged_load<T::Y_MN, !TN && !SWAP, PAIR, T::Y_ROWS>(dst + T::X_BYTES, &tmap_y, bar, y_mn,
                                                                               red + 64 * h, ti.g);
                        }
                        plain |= 1u << s;
                        uses ^= 1u << s;
                    }
                    ++it;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            // every copy issued lands before the CTA exits (a peer's copies
            // are counted on the leader's barriers; warp 2 waits for tails)
            if (leader) {
                const uint32_t n = it < stages ? it : stages;
                for (uint32_t i = it - n; i < it; ++i)
                    if ((plain >> (i % stages)) & 1u)
                        drain_ragged(&full[i % stages], ((uses >> (i % stages)) & 1) ^ 1, abort_flag, p);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if constexpr (F32)
            regs_dec<RAGGED_REGS_OTHER>();
        if (lane == 0 && leader) {
            const uint32_t base = smem_addr(smem);
            const uint64_t x0 = ragged_desc<T::X_MN>(base);
            const uint64_t y0 = ragged_desc<T::Y_MN>(base + T::X_BYTES);
            constexpr uint32_t X_STEP = (T::X_MN ? 2048u : 32u) >> 4; // 16 along the reduction
            constexpr uint32_t Y_STEP = (T::Y_MN ? 2048u : 32u) >> 4;
            uint32_t s = 0, phase = 0, tile_it = 0;
            uint32_t full_phase = 0, tail_phase = 0; // TN: per stage
            bool ok = true;
            for (int t = t_first; ok && t < num_tiles; t += t_stride) {
                const RaggedTile ti = ragged_tile<DIR, SWAP, T::BM, BN, T::BK>(p, t, group, tiles, first, count);
                const int nkb = SWAP ? kb_count : ti.nkb;
                if (nkb == 0)
                    continue;
                uint32_t buf = tile_it & 1;
                if (!wait_ragged(&acc_empty[buf], ((tile_it >> 1) & 1) ^ 1, abort_flag, p))
                    break;
                for (int kb = 0; kb < nkb; ++kb) {
                    // FP32 results: a fresh accumulator for each partial sum
                    if (F32 && kb > 0 && kb % PARTIAL == 0) {
                        buf = ++tile_it & 1;
                        if (!wait_ragged(&acc_empty[buf], ((tile_it >> 1) & 1) ^ 1, abort_flag, p)) {
                            ok = false;
                            break;
                        }
                    }
                    const uint32_t d = tmem_base + buf * (uint32_t)BN;
                    const bool first_kb = F32 ? kb % PARTIAL == 0 : kb == 0;
                    int steps = T::BK / 16;
                    if constexpr (TN) {
                        // a segment's last block is announced by warp 2
                        const bool tail = ti.rows - kb * T::BK < T::BK;
                        const uint32_t parity = ((tail ? tail_phase : full_phase) >> s) & 1;
                        // (a pair's is announced by both CTAs, each after writes to its own memory)
                        if (!(PAIR && tail ? wait_cluster(&tail_ready[s], parity, abort_flag, p)
                                           : wait_ragged(tail ? &tail_ready[s] : &full[s], parity, abort_flag, p))) {
                            ok = false;
                            break;
                        }
                        if (tail) {
                            tail_phase ^= 1u << s;
                            steps = (ti.rows - kb * T::BK + 15) / 16;
                        } else {
                            full_phase ^= 1u << s;
                        }
                    } else if (!wait_ragged(&full[s], phase, abort_flag, p)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t xd = x0 + s * (T::STAGE_BYTES >> 4);
                    const uint64_t yd = y0 + s * (T::STAGE_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < T::BK / 16; ++k)
                        if (!TN || k < steps)
                            mma_f16<PAIR>(d, xd + (k / 4) * (T::HALF_BYTES >> 4) + (k % 4) * X_STEP,
                                          yd + (k / 4) * (T::HALF_BYTES >> 4) + (k % 4) * Y_STEP, p.idesc,
                                          (!first_kb || k > 0) ? 1u : 0u);
                    if constexpr (PAIR)
                        mma_commit_pair_mc(&empty[s], 0x3);
                    else
                        mma_commit(&empty[s]);
                    if (kb == nkb - 1 || (F32 && kb % PARTIAL == PARTIAL - 1)) {
                        if constexpr (PAIR)
                            mma_commit_pair_mc(&acc_full[buf], 0x3);
                        else
                            mma_commit(&acc_full[buf]);
                    }
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                ++tile_it;
            }
            // all MMAs complete before tensor memory is released
            if constexpr (PAIR)
                mma_commit_pair(mma_done);
            else
                mma_commit(mma_done);
            drain_ragged(mma_done, 0, abort_flag, p);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ segment ends (TN)
        if constexpr (F32)
            regs_dec<RAGGED_REGS_OTHER>();
        // The last block of a segment holds rows of the next one (or behind
        // the last): they are cleared in both operands, so that they count as
        // zero whatever they hold.  A reduction row is one 128-byte line per
        // 64-element chunk, wherever the swizzle puts its pieces.
        if constexpr (TN) {
            uint32_t s = 0, tail_phase = 0;
            bool ok = true;
            for (int t = t_first; ok && t < num_tiles; t += t_stride) {
                const RaggedTile ti = ragged_tile<DIR, SWAP, T::BM, BN, T::BK>(p, t, group, tiles, first, count);
                s += (uint32_t)ti.nkb;
                while (s >= stages)
                    s -= stages;
                const int valid = ti.rows & (T::BK - 1);
                if (valid == 0)
                    continue;
                const uint32_t st = s == 0 ? stages - 1 : s - 1; // the segment's last block
                bool got = wait_ragged(&tail_full[st], (tail_phase >> st) & 1, abort_flag, p);
                if (!got) // aborting: an issued copy still lands before the CTA exits
                    drain_ragged(&tail_full[st], (tail_phase >> st) & 1, abort_flag, p);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tail_phase ^= 1u << st;
                constexpr int CHUNKS = (int)(T::HALF_BYTES / 8192);
                const int end = (valid + 15) & ~15; // the MMAs' steps of 16 end here
                const uint32_t at = smem_addr(smem) + st * T::STAGE_BYTES + (lane & 7) * 16;
                for (int r = valid + (lane >> 3); r < end; r += 4)
#pragma unroll
                    for (int c = 0; c < CHUNKS; ++c)
                        st_shared_v4(at + (r >> 6) * T::HALF_BYTES + c * 8192 + (r & 63) * 128, 0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        mbar_arrive_cluster_release(map_shared_rank(smem_addr(&tail_ready[st]), 0u));
                    else
                        mbar_arrive(&tail_ready[st]);
                }
            }
        }
    } else if (warp == 3) {
        if constexpr (F32)
            regs_dec<RAGGED_REGS_OTHER>();
        // ------------------------------------------------------------ hand-back of received sums (split)
        // The other CTAs' next writes come after this one's reads: a release at
        // cluster scope, by a warp that has no stores on their way.  From the
        // epilogue warps it would wait for those of the tile before (64 groups of
        // 8 rows, N = 2112, K = 2048, shared by 8: 235 -> 294 us).
        if (split) {
            uint32_t parity = 0;
            for (int t = t_first; t < num_tiles; t += t_stride, parity ^= 1u) {
                const bool got = wait_ragged(recv_read, parity, abort_flag, p);
                if (!__all_sync(0xffffffffu, got))
                    break;
                if (lane < p.split)
                    mbar_arrive_cluster_release(map_shared_rank(smem_addr(recv_free), (uint32_t)lane));
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if constexpr (F32) // these warps hold the sums
            regs_inc<RAGGED_REGS_EPILOGUE>();
        const int q = warp & 3;
        constexpr int NC = BN / 2; // columns of this warp, from c_first on
        const int c_first = warp >= 8 ? NC : 0;
        const uint32_t taddr0 = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c_first;
        const uint32_t stg_w =
            smem_addr(smem + p.off_out) + (uint32_t)(warp - 4) * (uint32_t)p.out_slots * RAGGED_SLOT_BYTES;
        const bool bf16 = p.out_type == RAGGED_OUT_BF16;
        uint32_t tile_it = 0, slot = 0;
        for (int t = t_first; t < num_tiles; t += t_stride) {
            const RaggedTile ti = ragged_tile<DIR, SWAP, T::BM, BN, T::BK>(p, t, group, tiles, first, count);
            const bool zero = ti.nkb == 0; // TN: a group without rows
            if (zero && p.accumulate)
                continue;
            if constexpr (F32) {
                // the tile's partial sums, added up in registers
                float acc[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    acc[c] = 0.0f;
                bool got = true;
                for (int kb = 0; kb < ti.nkb; kb += PARTIAL, ++tile_it) {
                    const uint32_t buf = tile_it & 1;
                    got = wait_ragged(&acc_full[buf], (tile_it >> 1) & 1, abort_flag, p);
                    got = __all_sync(0xffffffffu, got);
                    if (!got)
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < NC; c += 32) {
                        float v[32];
                        tmem_ld32(taddr0 + buf * (uint32_t)BN + c, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            acc[c + j] += v[j];
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR && !leader)
                            mbar_arrive_cluster(map_shared_rank(smem_addr(&acc_empty[buf]), 0u));
                        else
                            mbar_arrive(&acc_empty[buf]);
                    }
                }
                if (!got)
                    break;
                const int row = ti.i0 + (PAIR ? (int)rank * 128 : 0) + q * 32;
                if (row >= p.d_rows)
                    continue;
#pragma unroll
                for (int c = 0; c < NC; c += 32) {
                    const int col = ti.j0 + c_first + c;
                    if (col >= p.d_cols)
                        break;
                    if (lane == 0) { // the slot's last store has read it
                        if (p.out_slots == 2)
                            bulk_wait_read_1();
                        else
                            bulk_wait_read_all();
                    }
                    __syncwarp();
                    const uint32_t stg = stg_w + slot * RAGGED_SLOT_BYTES;
                    // 16-byte piece i of row r sits at piece i ^ (r % 8): TMA's 128-byte swizzle
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(stg + lane * 128 + ((i ^ (lane & 7)) << 4), __float_as_uint(acc[c + 4 * i]),
                                     __float_as_uint(acc[c + 4 * i + 1]), __float_as_uint(acc[c + 4 * i + 2]),
                                     __float_as_uint(acc[c + 4 * i + 3]));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (p.accumulate)
                            tma_add_3d(&tmap_d, stg, col, row, ti.g);
                        else
                            tma_store_3d(&tmap_d, stg, col, row, ti.g);
                        bulk_commit_group();
                    }
                    __syncwarp();
                    slot = slot + 1 == (uint32_t)p.out_slots ? 0 : slot + 1;
                }
                continue;
            }
            const uint32_t buf = tile_it & 1;
            if (!zero) {
                const bool got = wait_ragged(&acc_full[buf], (tile_it >> 1) & 1, abort_flag, p);
                if (!__all_sync(0xffffffffu, got))
                    break;
                tc_fence_after();
            }
            const uint32_t taddr = taddr0 + buf * (uint32_t)BN;
            const int i0 = ti.i0 + (PAIR ? (int)rank * 128 : 0) + q * 32; // this warp's first X row
            if constexpr (SWAP && BN <= RAGGED_SPLIT_MAX_BN) {
                if (split) {
                    const int tok_all = min(BN, ti.rows - ti.j0); // token rows of the tile,
                    const int shift = __ffs(BN / p.split) - 1;
                    const int own = 1 << shift; // of which every CTA owns so many
                    float v[32];
                    if constexpr (NC == 8)
                        tmem_ld8p(taddr, v);
                    else if constexpr (NC == 16)
                        tmem_ld16(taddr, v);
                    else
                        tmem_ld32(taddr, v);
                    tmem_wait_ld(v);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&acc_empty[buf]);
                    // what was sent for the tile before has been read everywhere
                    bool got = wait_cluster(recv_free, (tile_it & 1) ^ 1, abort_flag, p);
                    if (!__all_sync(0xffffffffu, got))
                        break;
                    // received: [source][owned token row][128 columns]
                    const uint32_t recv = smem_addr(smem + p.off_recv);
                    const uint32_t mine = recv + (uint32_t)((rank * own * 128 + q * 32 + lane) * 4);
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        const int tok = c_first + j;
                        if (tok < tok_all) {
                            const int to = tok >> shift;
                            st_cluster_f32(map_shared_rank(mine + (uint32_t)((tok - to * own) * 512), (uint32_t)to),
                                           v[j]);
                        }
                    }
                    __syncwarp();
                    if (lane < NC >> shift) // the owners of this warp's token rows
                        mbar_arrive_cluster_release(
                            map_shared_rank(smem_addr(recv_full), (uint32_t)((c_first >> shift) + lane)));
                    got = wait_cluster(recv_full, tile_it & 1, abort_flag, p);
                    if (!__all_sync(0xffffffffu, got))
                        break;
                    // the owned token rows: 256 threads, a column each, every other
                    // row.  Warp 3 hands the buffer back.
                    const int x = (int)threadIdx.x - 128;
                    const int col = ti.i0 + (x & 127);
                    float sum[BN / 4];
#pragma unroll
                    for (int i = 0; i < BN / 4; ++i) {
                        const int t0 = (x >> 7) + 2 * i;
                        sum[i] = 0.0f;
                        if (t0 < own)
                            for (int z = 0; z < p.split; ++z)
                                sum[i] += ld_shared_f32(recv + (uint32_t)(((z * own + t0) * 128 + (x & 127)) * 4));
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(recv_read);
#pragma unroll
                    for (int i = 0; i < BN / 4; ++i) {
                        const int t0 = (x >> 7) + 2 * i, tok = (int)rank * own + t0;
                        if (t0 < own && tok < tok_all && col < p.d_cols)
                            static_cast<uint16_t *>(p.d)[(size_t)(ti.first + ti.j0 + tok) * p.d_cols + col] =
                                (uint16_t)pack_16x2(sum[i], 0.0f, bf16);
                    }
                    ++tile_it;
                    continue;
                }
            }
            if constexpr (SWAP) {
                // a lane owns output column i0 + lane and the tile's token
                // rows: 32 lanes store 64 consecutive bytes of a row
                const int col = i0 + lane;
                const int tok = min(NC, ti.rows - ti.j0 - c_first);
                uint16_t *dst =
                    static_cast<uint16_t *>(p.d) + (size_t)(ti.first + ti.j0 + c_first) * p.d_cols + col;
                constexpr int W = NC < 32 ? NC : 32;
#pragma unroll
                for (int c = 0; c < NC; c += W) {
                    if (c >= tok)
                        break;
                    float v[W < 16 ? 16 : W];
                    if constexpr (W == 8)
                        tmem_ld8(taddr + c, v);
                    else if constexpr (W == 16)
                        tmem_ld16(taddr + c, v);
                    else
                        tmem_ld32(taddr + c, v);
                    tmem_wait_ld(v);
                    if (col < p.d_cols) {
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            if (c + j < tok)
                                dst[(size_t)(c + j) * p.d_cols] = (uint16_t)pack_16x2(v[j], 0.0f, bf16);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&acc_empty[buf]);
                ++tile_it;
                continue;
            }
            // rows of this warp that are stored: a segment may end inside the
            // tile (NT, NN); TN clips at the tensor's edge
            const int left = TN ? 32 : ti.rows - i0;
            const bool whole = TN || left >= 32;
            if (left <= 0) { // none: the warp hands the accumulator back unread
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && !leader)
                        mbar_arrive_cluster(map_shared_rank(smem_addr(&acc_empty[buf]), 0u));
                    else
                        mbar_arrive(&acc_empty[buf]);
                }
                ++tile_it;
                continue;
            }
            const int row = TN ? i0 : ti.first + i0;
            // columns of this warp that exist
            const int c_end = TN && row >= p.d_rows ? 0 : min(NC, p.d_cols - ti.j0 - c_first);
#pragma unroll 1
            for (int c = 0; c < NC; c += 64) {
                float v[2][32];
                if (c >= c_end) {
                    if (!zero && c + 64 >= NC) {
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR && !leader)
                                mbar_arrive_cluster(map_shared_rank(smem_addr(&acc_empty[buf]), 0u));
                            else
                                mbar_arrive(&acc_empty[buf]);
                        }
                    }
                    continue;
                }
                if (zero) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[0][j] = v[1][j] = 0.0f;
                } else {
                    tmem_ld32(taddr + c, v[0]);
                    tmem_ld32(taddr + c + 32, v[1]);
                    tmem_wait_ld(v[0]);
                    reg_tie32(v[1]);
                    if (c + 64 == NC) { // the warp has read its part of the accumulator
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR && !leader)
                                mbar_arrive_cluster(map_shared_rank(smem_addr(&acc_empty[buf]), 0u));
                            else
                                mbar_arrive(&acc_empty[buf]);
                        }
                    }
                }
                const int col = ti.j0 + c_first + c;
                // the slot's last store has read it
                if (lane == 0) {
                    if (p.out_slots == 2)
                        bulk_wait_read_1();
                    else
                        bulk_wait_read_all();
                }
                __syncwarp();
                const uint32_t stg = stg_w + slot * RAGGED_SLOT_BYTES;
                const uint32_t line = stg + lane * 128;
                // 16-byte piece i of row r sits at piece i ^ (r % 8): TMA's 128-byte swizzle
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *w = &v[i >> 2][(i & 3) * 8];
                    st_shared_v4(line + ((i ^ (lane & 7)) << 4), pack_16x2(w[0], w[1], bf16),
                                 pack_16x2(w[2], w[3], bf16), pack_16x2(w[4], w[5], bf16),
                                 pack_16x2(w[6], w[7], bf16));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (whole) {
                    if (lane == 0) {
                        if constexpr (TN)
                            tma_store_3d(&tmap_d, stg, col, row, ti.g);
                        else
                            tma_store_2d(&tmap_d, stg, col, row);
                        bulk_commit_group();
                    }
                } else {
                    // a segment's last rows: 8 lanes store a row's 128 bytes
                    const int piece = lane & 7;
#pragma unroll 1
                    for (int r = lane >> 3; r < left; r += 4) {
                        const uint4 w = ld_shared_v4(stg + r * 128 + ((piece ^ (r & 7)) << 4));
                        if (col + piece * 8 < p.d_cols)
                            st_global_v4(static_cast<uint16_t *>(p.d) + (size_t)(row + r) * p.d_cols + col + piece * 8,
                                         w.x, w.y, w.z, w.w);
                    }
                    if (lane == 0)
                        bulk_commit_group(); // empty: keeps one group per slot use
                }
                __syncwarp();
                slot = slot + 1 == (uint32_t)p.out_slots ? 0 : slot + 1;
            }
            if (!zero)
                ++tile_it;
        }
        // every store has completed before the CTA exits
        if (lane == 0)
            bulk_wait_all();
    }

    __syncwarp();
    if (PAIR || split)
        cluster_sync(); // no CTA leaves while another may still use its memory
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem_base, T::TMEM_COLS);
        else
            tmem_dealloc(tmem_base, T::TMEM_COLS);
    }
}

} // namespace fp8nt
