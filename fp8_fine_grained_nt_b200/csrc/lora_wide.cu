// Low-rank adapters of many requests, long batches: both products on the
// tensor cores in one kernel.
//
//   d[t, n] = c[t, n] + scale_g * sum_r v[t, r] B_g[n, r],   v[t, r] = sum_k x[t, k] A_g[r, k]
//
// A cluster of 1, 2, 4 or 8 CTAs takes 128 slots.  x, c and d are by far most
// of the bytes, so each is touched once: every CTA of the cluster reads a
// share of k of the slots' rows of x (v in FP32 in tensor memory), the shares
// are added up in order through distributed shared memory, and every CTA adds
// v B^T to a share of the columns.  v never leaves the SMs, and nothing needs
// a workspace.
//
//   phase 1   four warps gather the slots' rows of x into a ring (cp.async,
//             written in the layout the MMA reads), TMA brings A; M = 128
//             slots, N = rank.
//   exchange  each CTA puts its FP32 share of v into its shared memory; after
//             a cluster barrier every CTA adds the shares of its part of the
//             slots in rank order, splits v into two 16-bit terms and writes
//             them into every CTA's shared memory (hi + lo: 16 bits of
//             mantissa with BF16, 22 with FP16, so that the middle result
//             costs no accuracy; an FP16 row is divided by a power of two
//             first, so that v may exceed its range).
//   phase 2   128 columns at a time, hi B^T + lo B^T into one of two
//             accumulators; the epilogue adds c, which it fetched into shared
//             memory while the MMAs ran, rounds once and stores whole lines.
//
// Slots of more than one adapter: a pass over x handles four of them (one for
// ranks above 64) with their own accumulators; a slot's lane picks its own, so
// an adapter's Inf or NaN stays in its rows.  Slots sorted by adapter need one
// pass almost everywhere.
//
// 4096 rows of 8 adapters, rank 64, K = 7168, N = 4096: 40 us, where the bytes
// take 20.5 (clusters of 4 on 128 of the 148 SMs).  The phases follow one
// another: 1.6 us until the slots are known, 13.3 of reading x (4.4 TB/s), 6.3
// of exchange (two cluster barriers, reads and writes through distributed
// shared memory), 13.2 for c, d and the products (5.1 TB/s), and 4 between the
// last stores and the next call's start.  x comes by cp.async because TMA picks
// rows too slowly for 128 bytes of each: 80 cycles for four rows, 65 us in all.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "fp8_nt.h"
#include "grouped.h"
#include "kernel.cuh"
#include "lora_common.cuh"

namespace fp8nt {

namespace {

constexpr int WIDE_SLOTS = 128;
constexpr int WIDE_THREADS = 512;
constexpr int WIDE_WARPS = WIDE_THREADS / 32;
constexpr int WIDE_MAX_STAGES = 8;
constexpr uint32_t WIDE_X_BYTES = WIDE_SLOTS * 128; // 128 rows of 64 elements
constexpr uint32_t WIDE_B_BYTES = 128 * 128;        // 128 columns x 64 ranks
constexpr uint32_t WIDE_C_BYTES = WIDE_SLOTS * 256; // 128 slots x 128 columns

struct WidePlan {
    int cluster;
    int segs;        // adapters per pass
    int stages2;     // of the B ring
    uint32_t a_bytes; // 64 of k of one adapter's A
    uint32_t ring;    // bytes of the first ring: as many stages as a pass's adapters allow
    // in the room of the first ring, once phase 1 is done: the exchanged shares, and
    uint32_t off_c; // two c buffers: behind the shares, or in their place
    uint32_t off_v; // hi, lo: [2][rank chunk][128][128 B]
    uint32_t off_b; // B ring
    uint32_t off_bars;
    uint32_t total;
};

struct WideParams {
    LoraParams p;
    WidePlan plan;
    uint32_t idesc; // of the MMAs, without the number of columns
    uint64_t timeout_ns;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, bool in)
{
    // (a source size of 0 fills the 16 bytes with zeros)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// At most n, up to 6, of the thread's groups are still on their way.
__device__ __forceinline__ void cp_async_wait_for(int n)
{
    switch (n) {
    case 0: cp_async_wait<0>(); break;
    case 1: cp_async_wait<1>(); break;
    case 2: cp_async_wait<2>(); break;
    case 3: cp_async_wait<3>(); break;
    case 4: cp_async_wait<4>(); break;
    case 5: cp_async_wait<5>(); break;
    default: cp_async_wait<6>(); break;
    }
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Bit i: one of the warp's slots belongs to adapter i of the pass.
__device__ __forceinline__ uint32_t segments_present(int mine, int segs)
{
    return __reduce_or_sync(0xffffffffu, mine >= 0 && mine < segs ? 1u << mine : 0u);
}

template <bool BF16>
__global__ void __launch_bounds__(WIDE_THREADS, 1)
    lora_wide_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ WideParams wp)
{
    const LoraParams &p = wp.p;
    const WidePlan &plan = wp.plan;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem =
        reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *full1 = reinterpret_cast<uint64_t *>(smem + plan.off_bars); // x and A of a stage are there
    uint64_t *empty1 = full1 + WIDE_MAX_STAGES;
    uint64_t *full2 = empty1 + WIDE_MAX_STAGES; // B of a stage is there
    uint64_t *empty2 = full2 + WIDE_MAX_STAGES;
    uint64_t *p1_done = empty2 + WIDE_MAX_STAGES; // this CTA's share of v is complete
    uint64_t *acc_full = p1_done + 1;             // accumulator complete (x2)
    uint64_t *acc_empty = acc_full + 2;           // accumulator read (x2)
    uint64_t *mma_done = acc_empty + 2;
    __shared__ uint32_t tmem_slot;
    __shared__ uint32_t abort_word;
    __shared__ int slot_row[WIDE_SLOTS], slot_seg[WIDE_SLOTS]; // row; segment, -1 without an adapter
    __shared__ int seg_adapter[WIDE_SLOTS];
    __shared__ uint32_t warp_starts[4]; // slots of 32 at which a segment starts
    __shared__ float adapter_scale[WIDE_SLOTS], slot_scale[WIDE_SLOTS]; // scale_g; times the power of two
    volatile uint32_t *abort_flag = &abort_word;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        const uint32_t a = smem_addr(bar);
        return mbar_try_wait(a, parity) || wait_slow(a, parity, abort_flag, p.status, wp.timeout_ns, true);
    };

    // ---------------------------------------------------------------- set-up
    if (tid == 0) {
        for (int s = 0; s < WIDE_MAX_STAGES; ++s) {
            mbar_init(&full1[s], 4 + 1); // the gathering warps and the TMA thread
            mbar_init(&empty1[s], 1);
            mbar_init(&full2[s], 1);
            mbar_init(&empty2[s], 1);
        }
        mbar_init(p1_done, 1);
        mbar_init(mma_done, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        abort_word = 0u;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_b);
    }
    if (warp == 4) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const int slot0 = blockIdx.y * WIDE_SLOTS;
    // the block's slots and their segments (runs of one adapter)
    Slot mine = {-1, -1};
    if (warp < 4) {
        mine = read_slot(p, slot0 + tid);
        slot_row[tid] = mine.row;
        slot_seg[tid] = mine.adapter;
    }
    __syncthreads();
    const bool starts = warp < 4 && mine.adapter >= 0 && (tid == 0 || slot_seg[tid - 1] != mine.adapter);
    const uint32_t start_mask = __ballot_sync(0xffffffffu, starts);
    if (warp < 4 && lane == 0)
        warp_starts[warp] = start_mask;
    __syncthreads();
    if (warp < 4) {
        int seg = __popc(start_mask & (0xffffffffu >> (31 - lane))) - 1;
        for (int w = 0; w < warp; ++w)
            seg += __popc(warp_starts[w]);
        slot_seg[tid] = mine.adapter >= 0 ? seg : -1;
        if (starts)
            seg_adapter[seg] = mine.adapter;
    }
    // (needed in the exchange)
    const float scale = mine.adapter >= 0 ? __ldg(p.scales + mine.adapter) : 0.0f;
    tc_fence_before();
    cluster_arrive_relaxed(); // (all of the cluster runs before any shared memory of another CTA is touched)
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int cl = plan.cluster;
    const int rank = (int)cluster_ctarank();
    const int total_segs =
        __popc(warp_starts[0]) + __popc(warp_starts[1]) + __popc(warp_starts[2]) + __popc(warp_starts[3]);
    // this CTA's shares: every cl-th block of k and of columns, so that the
    // cluster as a whole reads and writes long runs of each row (kbs below)
    const int n_tiles = ((p.N + 127) / 128 - rank + cl - 1) / cl;
    const int chunks = (p.R + 63) / 64;
    const int ranks = (p.R + 15) / 16 * 16; // columns of an adapter in phase 1
    const int pitch = p.R + 4; // floats per row of the exchanged shares

    // ring positions, kept over the passes by each role
    uint32_t it2 = 0, pass_it = 0;
    uint32_t acc_phase = 0; // bit b: parity of accumulator b
    uint32_t phase1 = 0; // bit s: parity of stage s of the first ring (the ring restarts with each pass)
    const uint32_t s2 = (uint32_t)plan.stages2;
    bool ok = true;
    cluster_wait();

    for (int seg0 = 0; seg0 < total_segs; seg0 += plan.segs, ++pass_it) {
        const int segs = min(plan.segs, total_segs - seg0);
        const uint32_t stage_bytes = WIDE_X_BYTES + (uint32_t)segs * plan.a_bytes; // 64 of k
        const int kbs = ((p.K + 63) / 64 - rank + cl - 1) / cl;
        const int s1 = min(WIDE_MAX_STAGES, (int)(plan.ring / stage_bytes)); // at least 4
        // a walk along the first ring: stage, and which of its uses in this pass is odd
        struct Ring {
            int s, stages;
            uint32_t odd;
            __device__ __forceinline__ void skip(int n)
            {
                s += n;
                while (s >= stages) {
                    s -= stages;
                    odd ^= 1u;
                }
            }
        };
        auto parity1 = [&](const Ring &r) { return ((phase1 >> r.s) ^ r.odd) & 1u; };
        auto load_b = [&](int t, int i, int rc) { // stage it2 of the B ring
            const uint32_t s = it2 % s2; // (of the B ring)
            if (!ok || !(ok = wait(&empty2[s], ((it2 / s2) & 1) ^ 1)))
                return;
            mbar_arrive_expect_tx(&full2[s], WIDE_B_BYTES);
            tma_load_nd<true, false>(smem + plan.off_b + s * WIDE_B_BYTES, &tmap_b, smem_addr(&full2[s]), rc * 64,
                                     (t * cl + rank) * 128, seg_adapter[seg0 + i]);
            ++it2;
        };
        // accumulators: two while a pass has at most two adapters (512 columns
        // of tensor memory), else one
        auto acc_buf = [&](int t) { return segs <= 2 ? t & 1 : 0; };
        auto acc_parity = [&](int t) { return ((acc_phase >> acc_buf(t)) ^ (uint32_t)(segs <= 2 ? t >> 1 : t)) & 1u; };
        const int b_loads = n_tiles * segs * chunks;
        int b_done = 0;

        // ------------------------------------------------------------ phase 1
        if (warp < 4) {
            // thread: 16-byte piece lane % 8 of rows 32 warp + 4 j + lane / 8
            const int piece = lane & 7;
            const uint16_t *src[8];
            uint32_t live = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = warp * 32 + 4 * j + (lane >> 3);
                const int seg = slot_seg[r];
                const bool in = seg >= seg0 && seg < seg0 + segs;
                src[j] = static_cast<const uint16_t *>(p.x) + (in ? slot_row[r] * p.ld_x : 0) + piece * 8;
                live |= (in ? 1u : 0u) << j;
            }
            const uint32_t dst = (uint32_t)((warp * 32 + (lane >> 3)) * 128);
            // a stage is published once its copies have landed, `lag` rounds
            // after they were issued
            const int lag = s1 >= 6 ? s1 - 2 : 3; // less than the stages there are
            Ring at = {0, s1, 0u}, behind = {0, s1, 0u};
            auto publish = [&]() {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&full1[behind.s]);
                behind.skip(1);
            };
            for (int i = 0; ok && i < kbs; ++i, at.skip(1)) {
                ok = wait(&empty1[at.s], parity1(at) ^ 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                const uint32_t to = base + at.s * stage_bytes + dst;
                const int k = (i * cl + rank) * 64;
                const bool k_in = k + piece * 8 < p.K;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = 4 * j + (lane >> 3); // (its low 3 bits are the row's)
                    const bool in = k_in && ((live >> j) & 1u);
                    cp_async_16(to + j * 512 + ((piece ^ (r & 7)) << 4),
                                in ? src[j] + k : static_cast<const uint16_t *>(p.x), in);
                }
                cp_async_commit();
                if (i >= lag) {
                    cp_async_wait_for(lag);
                    publish();
                }
            }
            for (int i = min(lag, kbs); ok && i > 0; --i) {
                cp_async_wait_for(i - 1);
                publish();
            }
            cp_async_wait<0>();
            adapter_scale[tid] = scale; // (read in the exchange)
        } else if (warp == 5) {
            if (lane == 0) {
                Ring at = {0, s1, 0u};
                for (int i = 0; ok && i < kbs; ++i, at.skip(1)) {
                    const int s = at.s;
                    if (!(ok = wait(&empty1[s], parity1(at) ^ 1u)))
                        break;
                    mbar_arrive_expect_tx(&full1[s], (uint32_t)segs * plan.a_bytes);
                    for (int j = 0; j < segs; ++j)
                        tma_load_nd<true, false>(smem + s * stage_bytes + WIDE_X_BYTES + j * plan.a_bytes, &tmap_a,
                                                 smem_addr(&full1[s]), (i * cl + rank) * 64, 0,
                                                 seg_adapter[seg0 + j]);
                }
                // the first stages of B, during the exchange
                ok = ok && wait(p1_done, pass_it & 1);
                for (; ok && b_done < min(b_loads, (int)s2); ++b_done)
                    load_b(b_done / (segs * chunks), b_done / chunks % segs, b_done % chunks);
            }
        } else if (warp == 4) {
            if (lane == 0) {
                const uint32_t idesc1 = wp.idesc | (uint32_t)(segs * ranks >> 3) << 17;
                Ring at = {0, s1, 0u};
                for (int i = 0; ok && i < kbs; ++i, at.skip(1)) {
                    const int s = at.s;
                    if (!(ok = wait(&full1[s], parity1(at))))
                        break;
                    tc_fence_after();
                    const uint64_t xd = make_sdesc(base + s * stage_bytes);
                    const uint64_t ad = make_sdesc(base + s * stage_bytes + WIDE_X_BYTES);
#pragma unroll
                    for (int k = 0; k < 4; ++k) // all adapters of the pass side by side
                        mma_f16<false>(tmem, xd + 2 * k, ad + 2 * k, idesc1, (i > 0 || k > 0) ? 1u : 0u);
                    mma_commit(&empty1[s]);
                }
                mma_commit(p1_done);
            }
        } else if (warp >= 8) {
            // this CTA's share of v: lane = slot
            const int q = warp & 3, r = q * 32 + lane;
            ok = wait(p1_done, pass_it & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc_fence_after();
                const int mine = slot_seg[r] - seg0;
                const uint32_t present = segments_present(mine, segs);
                const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
                const bool none = kbs <= 0; // more CTAs than blocks of k
                for (int c = (warp >= 12 ? 16 : 0); c < p.R; c += 32) { // two warps per 32 slots
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = 0.0f;
                    for (uint32_t left = present; left; left &= left - 1) {
                        const int i = __ffs(left) - 1;
                        float w[16];
                        tmem_ld16(taddr + i * ranks + c, w);
                        tmem_wait_ld(w);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = mine == i ? w[j] : v[j];
                    }
                    const uint32_t to = base + (uint32_t)(r * pitch + c) * 4u;
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        if (c + j < p.R)
                            st_shared_v4(to + j * 4, none ? 0u : __float_as_uint(v[j]),
                                         none ? 0u : __float_as_uint(v[j + 1]), none ? 0u : __float_as_uint(v[j + 2]),
                                         none ? 0u : __float_as_uint(v[j + 3]));
                }
                tc_fence_before();
            }
        }
        __syncwarp();

        // ------------------------------------------------------------ exchange
        // An epilogue warp has 32 slots and half of a tile's columns; its lanes
        // move whole 128-byte lines of c and d, 8 lanes each: slots er + 4 i +
        // lane / 8.  The first tile's c is on its way during the exchange where
        // its buffers lie behind the shares.
        const int er = (warp & 3) * 32, half = warp >= 12 ? 1 : 0;
        int rows[8]; // -1: not in this pass
        if (warp >= 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = er + 4 * i + (lane >> 3);
                const int seg = slot_seg[r];
                rows[i] = seg >= seg0 && seg < seg0 + segs ? slot_row[r] : -1;
            }
        }
        const int piece = half * 8 + (lane & 7); // of a slot's 16 pieces of 16 bytes
        // piece i of slot r in buffer b, spread over the banks
        auto c_at = [&](int b, int r, int i) {
            return base + plan.off_c + (uint32_t)(b * WIDE_C_BYTES + r * 256 + ((i ^ (r & 7)) << 4));
        };
        auto fetch_c = [&](int t) {
            const int col = (t * cl + rank) * 128 + piece * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (rows[i] >= 0 && col < p.N)
                    cp_async_16(c_at(t & 1, er + 4 * i + (lane >> 3), piece),
                                static_cast<const uint16_t *>(p.c) + (long)rows[i] * p.ld_c + col, true);
            cp_async_commit();
        };
        const bool early = plan.off_c > 0;
        cluster_arrive(); // before the copies of c: a release would wait for them, 2 us
        if (early && warp >= 8 && n_tiles > 0)
            fetch_c(0);
        cluster_wait(); // every CTA's share is there
        // this CTA's part of the slots, two per round of a warp
        const int part = WIDE_SLOTS / cl;
        for (int i = warp; i < part; i += 2 * WIDE_WARPS) {
            const int rk = lane * 4;
            float4 v[2][8];
            int seg[2], r[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                r[h] = rank * part + i + h * WIDE_WARPS;
                seg[h] = i + h * WIDE_WARPS < part ? slot_seg[r[h]] : -1;
                if (seg[h] < seg0 || seg[h] >= seg0 + segs)
                    seg[h] = -1;
                const uint32_t at = base + (uint32_t)(r[h] * pitch + rk) * 4u;
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    v[h][z] = z < cl && seg[h] >= 0 && rk < p.R ? ld_shared_cluster_v4(map_shared_rank(at, (uint32_t)z))
                                                               : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (seg[h] < 0)
                    continue;
                float4 sum = v[h][0];
#pragma unroll
                for (int z = 1; z < 8; ++z) {
                    sum.x += v[h][z].x;
                    sum.y += v[h][z].y;
                    sum.z += v[h][z].z;
                    sum.w += v[h][z].w;
                }
                float power = 1.0f;
                if constexpr (!BF16)
                    power = lora_fp16_scale(
                        fmaxf(fmaxf(fabsf(sum.x), fabsf(sum.y)), fmaxf(fabsf(sum.z), fabsf(sum.w))));
                const float inv = 1.0f / power; // a power of two: exact
                uint32_t hi[2], lo[2];
                split_two<BF16>(sum.x * inv, sum.y * inv, hi[0], lo[0]);
                split_two<BF16>(sum.z * inv, sum.w * inv, hi[1], lo[1]);
                const uint32_t at = base + plan.off_v + (uint32_t)((rk >> 6) * WIDE_X_BYTES + r[h] * 128 +
                                                                   ((((rk & 63) >> 3) ^ (r[h] & 7)) << 4) + (rk & 7) * 2);
                const float f = power * adapter_scale[r[h]];
                for (int z = 0; z < cl; ++z) {
                    if (rk < chunks * 64) {
                        const uint32_t to = map_shared_rank(at, (uint32_t)z);
                        st_cluster_v2(to, hi[0], hi[1]);
                        st_cluster_v2(to + chunks * WIDE_X_BYTES, lo[0], lo[1]);
                    }
                    if (lane == 0)
                        st_cluster_f32(map_shared_rank(smem_addr(&slot_scale[r[h]]), (uint32_t)z), f);
                }
            }
        }
        fence_proxy_async_smem();
        cluster_sync(); // v is in every CTA, and nobody reads the shares any more
        fence_proxy_async_smem();
        if (!early && warp >= 8 && n_tiles > 0)
            fetch_c(0);

        // ------------------------------------------------------------ phase 2
        if (warp == 5) {
            if (lane == 0)
                for (; ok && b_done < b_loads; ++b_done)
                    load_b(b_done / (segs * chunks), b_done / chunks % segs, b_done % chunks);
        } else if (warp == 4) {
            if (lane == 0) {
                tc_fence_after();
                for (int t = 0; ok && t < n_tiles; ++t) {
                    const int buf = acc_buf(t);
                    if (!(ok = wait(&acc_empty[buf], acc_parity(t) ^ 1u)))
                        break;
                    for (int i = 0; ok && i < segs;) {
                        const uint32_t d = tmem + (buf * segs + i) * 128;
                        // two adapters at once where their B lies side by side
                        const int both = it2 % 2 == 0 && chunks == 1 && i + 1 < segs ? 2 : 1;
                        const uint32_t idesc2 = wp.idesc | (uint32_t)(both * 128 >> 3) << 17;
                        for (int rc = 0; ok && rc < chunks; ++rc, it2 += both) {
                            const uint32_t s = it2 % s2;
                            ok = wait(&full2[s], (it2 / s2) & 1);
                            if (both == 2)
                                ok = ok && wait(&full2[s + 1], (it2 / s2) & 1);
                            if (!ok)
                                break;
                            tc_fence_after();
                            const uint64_t bd = make_sdesc(base + plan.off_b + s * WIDE_B_BYTES);
                            const int steps = min(4, (p.R - rc * 64 + 15) / 16);
#pragma unroll
                            for (int term = 0; term < 2; ++term) {
                                const uint64_t vd =
                                    make_sdesc(base + plan.off_v + (uint32_t)(term * chunks + rc) * WIDE_X_BYTES);
                                for (int k = 0; k < steps; ++k)
                                    mma_f16<false>(d, vd + 2 * k, bd + 2 * k, idesc2,
                                                   (rc > 0 || term > 0 || k > 0) ? 1u : 0u);
                            }
                            mma_commit(&empty2[s]);
                            if (both == 2)
                                mma_commit(&empty2[s + 1]);
                        }
                        i += both;
                    }
                    mma_commit(&acc_full[buf]);
                }
            }
        } else if (warp >= 8) {
            const int q = warp & 3, r = q * 32 + lane;
            const int mine = slot_seg[r] - seg0;
            const uint32_t present = segments_present(mine, segs);
            const float f = (mine >= 0 && mine < segs) ? slot_scale[r] : 0.0f;
            for (int t = 0; t < n_tiles; ++t) {
                if (t + 1 < n_tiles) {
                    fetch_c(t + 1);
                    cp_async_wait<1>();
                } else {
                    cp_async_wait<0>();
                }
                __syncwarp(); // every lane's pieces of c are there
                const int buf = acc_buf(t);
                ok = wait(&acc_full[buf], acc_parity(t));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + buf * segs * 128 + half * 64;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    float v[32];
                    for (uint32_t left = present; left; left &= left - 1) {
                        const int i = __ffs(left) - 1;
                        if (left == present) { // the first, usually the only one
                            tmem_ld32(taddr + i * 128 + c, v);
                            tmem_wait_ld(v);
                        } else {
                            float w[32];
                            tmem_ld32(taddr + i * 128 + c, w);
                            tmem_wait_ld(w);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = mine == i ? w[j] : v[j];
                        }
                    }
                    if (c == 32) { // the accumulator has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        const uint32_t at = c_at(t & 1, r, half * 8 + ((c + j) >> 3));
                        const uint4 in = ld_shared_v4(at);
                        const uint32_t old[4] = {in.x, in.y, in.z, in.w};
                        uint32_t out[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 o = unpack2<BF16>(old[i]);
                            out[i] = pack2<BF16>(fmaf(f, v[j + 2 * i], o.x), fmaf(f, v[j + 2 * i + 1], o.y));
                        }
                        st_shared_v4(at, out[0], out[1], out[2], out[3]);
                    }
                }
                __syncwarp();
                const int col = (t * cl + rank) * 128 + piece * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (rows[i] >= 0 && col < p.N) {
                        const uint4 o = ld_shared_v4(c_at(t & 1, er + 4 * i + (lane >> 3), piece));
                        st_global_v4(static_cast<uint16_t *>(p.d) + (long)rows[i] * p.ld_d + col, o.x, o.y, o.z, o.w);
                    }
                __syncwarp();
            }
            cp_async_wait<0>();
        }
        __syncwarp();
        for (int s = 0; s < s1 && s < kbs; ++s)
            phase1 ^= (uint32_t)((kbs - s + s1 - 1) / s1 & 1) << s;
        if (segs <= 2)
            acc_phase ^= (uint32_t)((n_tiles + 1) >> 1 & 1) | (uint32_t)(n_tiles >> 1 & 1) << 1;
        else
            acc_phase ^= (uint32_t)(n_tiles & 1);
        // ordinary accesses of the rings come before the next pass's TMA writes
        fence_proxy_async_smem();
        __syncthreads();
    }

    // all MMAs complete before tensor memory is released; where a wait ran out,
    // copies that nothing waited for land before the CTA exits
    if (warp == 4 && lane == 0) {
        mma_commit(mma_done);
        const uint32_t a = smem_addr(mma_done);
        if (!mbar_try_wait(a, 0))
            wait_slow(a, 0, abort_flag, p.status, wp.timeout_ns, false);
        if (*abort_flag) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
    }
    cluster_sync(); // nobody leaves while another CTA may still use its shared memory
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Shared memory of a call: see the kernel's phases.
WidePlan wide_plan(int slots, int R, int sms)
{
    WidePlan w = {};
    const int blocks = (slots + WIDE_SLOTS - 1) / WIDE_SLOTS;
    // as many CTAs per block of slots as run at once
    w.cluster = 8;
    while (w.cluster > 1 && (w.cluster > sms || blocks > clusters_held(w.cluster, sms)))
        w.cluster /= 2;
    const uint32_t chunks = (uint32_t)(R + 63) / 64;
    w.segs = R <= 64 ? 4 : 1;
    w.a_bytes = (uint32_t)(R + 15) / 16 * 16 * 128;
    // Phase 1 waits for memory (about 2.6 us a round trip under load), so its ring
    // has all the room: eight stages of 64 of k with one adapter up to rank 64,
    // six with two, or with one above, four with four.  Of phase 2, the c buffers
    // lie behind the shares up to rank 64, else in their place.
    const uint32_t shares = align_up_u32((uint32_t)WIDE_SLOTS * (uint32_t)(R + 4) * 4u, 1024);
    w.off_c = R <= 64 ? shares : 0;
    w.off_v = w.off_c + 2 * WIDE_C_BYTES > shares ? w.off_c + 2 * WIDE_C_BYTES : shares;
    w.off_b = w.off_v + 2 * chunks * WIDE_X_BYTES;
    // two adapters' tiles take two stages of B, the next tile's two more
    w.stages2 = R <= 64 ? 4 : 5;
    w.ring = w.off_b + (uint32_t)w.stages2 * WIDE_B_BYTES;
    const uint32_t least = 4u * (WIDE_X_BYTES + 4u * 64u * 128u); // four stages of four adapters of rank 64
    w.ring = w.ring > least ? w.ring : least;
    w.off_bars = w.ring;
    w.total = w.off_bars + 8u * (4u * WIDE_MAX_STAGES + 6u);
    return w;
}

template <bool BF16>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const WideParams &wp, const DeviceView &dev,
                   cudaStream_t stream)
{
    // under a bound on the SMs, as many blocks of slots at a time as go into it
    // (and no overlap of the launches)
    const int most = clusters_held(wp.plan.cluster, dev.sms) * WIDE_SLOTS;
    if (dev.bounded && wp.p.slots > most) {
        cudaError_t err = cudaSuccess;
        for (int first = 0; err == cudaSuccess && first < wp.p.slots; first += most) {
            WideParams piece = wp;
            piece.p = lora_piece(wp.p, first, min(most, wp.p.slots - first));
            err = launch<BF16>(ta, tb, piece, dev, stream);
        }
        return err;
    }
    static std::atomic<bool> ready[64];
    auto kernel = lora_wide_kernel<BF16>;
    const int smem = (int)wp.plan.total + 1024;
    if (!ready[dev.index].load(std::memory_order_acquire)) {
        const cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem - 4096);
        if (err != cudaSuccess)
            return err;
        ready[dev.index].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)wp.plan.cluster, (unsigned)((wp.p.slots + WIDE_SLOTS - 1) / WIDE_SLOTS), 1);
    cfg.blockDim = dim3(WIDE_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)wp.plan.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dev.bounded ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, ta, tb, wp);
}

} // namespace

// Long batches with enough slots per adapter; grid.y counts blocks of slots.
// Measured, short form against this one, us from graphs (N = 4096, K = 7168, rank
// 64 but where said):
//                     256 rows   512      768      1024     2048     4096
//   1 adapter         16, 23     20, 23   26, 23   29, 24   51, 34    99, 36
//   8 adapters        16, 31     20, 23   26, 23   29, 24   52, 34   102, 37
//   8 of rank 16       9, 25     14, 22   16, 22   19, 22   31, 32    60, 35
//   2 of rank 128     20, 28     27, 28   36, 29   43, 29   84, 42   162, 45
//   32 rows of each   16, 31     20, 31   26, 31   32, 32   60, 53   111, 65
// One limit for all of them: it loses up to a fifth between 513 and 768 slots at
// ranks above 64 and between 769 and 2000 at rank 16.
// The host knows the adapters loaded, not those in use: an unsorted batch of many
// would make up to 32 passes (128 above rank 64) over each block of slots.  So a
// few adapters of a large pool take the short form too: 4096 rows of 8 adapters
// 38 us with up to 128 loaded, 101 with more (of 129 in use 155, of 128 65).
bool lora_is_wide(int slots, int adapters, int R)
{
    return slots > 768 && R <= 128 && slots / adapters >= 32 && slots <= 65535 * WIDE_SLOTS;
}

int launch_lora_wide(const LoraParams &p, bool bf16, const DeviceView &dev, cudaStream_t stream)
{
    WideParams wp;
    memset(&wp, 0, sizeof(wp));
    wp.p = p;
    wp.plan = wide_plan(p.slots, p.R, dev.sms);
    if ((int)wp.plan.total + 1024 > dev.max_smem - 4096)
        return DG_ERR_UNSUPPORTED_SHAPE;
    const int ranks = (p.R + 15) / 16 * 16;
    wp.idesc = ragged_idesc(bf16, false, false, 128, 0);
    wp.timeout_ns = dev.timeout_ns;
    const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap ta, tb;
    {
        const uint64_t dims[3] = {(uint64_t)p.K, (uint64_t)p.R, (uint64_t)p.adapters};
        const uint64_t strides[2] = {(uint64_t)p.K * 2, (uint64_t)p.R * (uint64_t)p.K * 2};
        const uint32_t box[3] = {64, (uint32_t)ranks, 1};
        const int st = make_tmap_128b(&ta, p.lora_a, type, 3, dims, strides, box);
        if (st != DG_OK)
            return st;
    }
    {
        const uint64_t dims[3] = {(uint64_t)p.R, (uint64_t)p.N, (uint64_t)p.adapters};
        const uint64_t strides[2] = {(uint64_t)p.R * 2, (uint64_t)p.N * (uint64_t)p.R * 2};
        const uint32_t box[3] = {64, 128, 1};
        const int st = make_tmap_128b(&tb, p.lora_b, type, 3, dims, strides, box);
        if (st != DG_OK)
            return st;
    }
    const cudaError_t err = bf16 ? launch<true>(ta, tb, wp, dev, stream) : launch<false>(ta, tb, wp, dev, stream);
    return err == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

} // namespace fp8nt
