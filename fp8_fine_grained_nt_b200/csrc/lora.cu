// Low-rank adapters of many requests beside a shared projection:
//
//   d[t, n] = c[t, n] + scale_g * sum_r v[t, r] B_g[n, r],   v[t, r] = sum_k x[t, k] A_g[r, k]
//
// for every slot i with adapter g = m_indices[i] and row t = order[i].  Slots
// sorted by adapter (as group_rows_by_index leaves them) share the reads of
// its weights.
//
// For short batches (lora_is_wide has the rule): one token to a few hundred.
// Both factors are thin, so neither bytes (1.5 us for 64 rows of 28 adapters,
// rank 16, K = 2048, N = 7168) nor products bound the operator but the latency
// of its chain: slots, loads, sums, v out and in again, loads, stores.  It
// takes 8.4 us a call there and 6 for one row (replayed from a graph, as all
// times in this file; 64 rows given by an index, of 32 adapters or none, 10.2).
// So the work is cut into about four CTAs per SM, every load is issued as early
// as its address is known, and the products run on operands loaded straight
// from global memory into registers (a 16-byte load gives a lane of the first
// kernel 8 consecutive elements of the reduction, which any pairing of
// mma.sync's k positions may use as long as both operands use the same one).
// Two kernels, the second set up while the first runs:
//   down  v in FP32 for a range of k per CTA (`splits` ranges, written side by
//         side: summed in order by the second kernel, so no atomics)
//   up    sums the ranges and adds v B^T to c, rounding once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "grouped.h"
#include "lora_common.cuh"

namespace fp8nt {

namespace {

constexpr int LORA_THREADS = 256;
constexpr int LORA_WARPS = 8;
constexpr int LORA_SLOTS = 16;   // slots per CTA of the first kernel: one MMA's rows
constexpr int LORA_UP_SLOTS = 8; // of the second
// Largest rank whose second product is done in FP32 (64 rows of 28 adapters, N =
// 7168, K = 2048: rank 8 7.7 us, with mma.sync 9.7; rank 16 8.4 and 9.5; rank 32
// 12.8 and 10.5).
constexpr int LORA_FP32_RANK = 16;

// bytes of v's sums, or of their shares
__host__ __device__ constexpr int lora_up_part(int R)
{
    return LORA_UP_SLOTS * R > LORA_THREADS * 4 ? LORA_UP_SLOTS * R * 4 : LORA_THREADS * 16;
}

// 16 x 8 += 16 x 16 * (8 x 16)^T, 16-bit operands, FP32 sums
template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bit i: a segment (run of one adapter) begins at slot i of a warp's slots, one
// slot per lane of the lowest `n` lanes.
__device__ __forceinline__ uint32_t segment_starts(int adapter, int lane, int n)
{
    const int before = __shfl_up_sync(0xffffffffu, adapter, 1);
    return __ballot_sync(0xffffffffu, lane < n && (lane == 0 || adapter != before));
}

// ---------------------------------------------------------------- down

// 16 slots, 8 NT ranks and one k range per CTA; a warp's job is one segment and
// a slice of the range (all of it once there are 8 segments or more).
template <bool BF16, int NT>
__global__ void __launch_bounds__(LORA_THREADS) lora_down_kernel(const LoraParams p)
{
    constexpr int SB = LORA_SLOTS;
    constexpr int RB = 8 * NT; // ranks of this CTA
    __shared__ float4 red[LORA_WARPS * SB * RB / 4]; // [slice][slot][rank]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane & 3, q = lane >> 2;
    grid_dependency_wait();
    grid_launch_dependents();
    const int slot0 = blockIdx.x * SB;
    const int r0 = (blockIdx.y + p.rank_block) * RB;
    const Slot mine = read_slot(p, lane < SB ? slot0 + lane : p.slots);
    const uint32_t starts = segment_starts(mine.adapter, lane, SB);
    const int segs = __popc(starts);
    const int slices = max(1, LORA_WARPS / segs);
    // (the end of a range is taken from what is left: K and N may be near 2^31)
    const int k_lo = blockIdx.z * p.k_chunk, k_hi = k_lo + min(p.k_chunk, p.K - k_lo);
    const int k_step = ((k_hi - k_lo + slices - 1) / slices + 31) / 32 * 32;

    for (int job = warp; job < segs * slices; job += LORA_WARPS) {
        const int seg = job / slices, ks = job % slices;
        uint32_t left = starts;
        for (int i = 0; i < seg; ++i)
            left &= left - 1;
        const int s0 = __ffs(left) - 1;
        left &= left - 1;
        const int s1 = left ? __ffs(left) - 1 : SB;
        const int g = __shfl_sync(0xffffffffu, mine.adapter, s0);
        if (g < 0)
            continue;
        // slots outside the segment and ranks past R read a row that is there:
        // their products are not used
        const int ka = k_lo + ks * k_step, kb = min(ka + k_step, k_hi);
        const uint16_t *xrow[2], *arow[NT];
        const int first_row = __shfl_sync(0xffffffffu, mine.row, s0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = h * 8 + q;
            const int row = __shfl_sync(0xffffffffu, mine.row, s);
            xrow[h] = static_cast<const uint16_t *>(p.x) + (size_t)(s >= s0 && s < s1 ? row : first_row) * p.ld_x +
                      ka + t * 8;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
            arow[j] = static_cast<const uint16_t *>(p.lora_a) + ((size_t)g * p.R + min(r0 + 8 * j + q, p.R - 1)) * p.K +
                      ka + t * 8;
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[j][e] = 0.0f;
        auto step = [&](bool in) {
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            uint4 xv[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                xv[h] = in ? __ldg(reinterpret_cast<const uint4 *>(xrow[h])) : zero;
                xrow[h] += 32;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 av = in ? __ldg(reinterpret_cast<const uint4 *>(arow[j])) : zero;
                arow[j] += 32;
                mma_16816<BF16>(acc[j], xv[0].x, xv[1].x, xv[0].y, xv[1].y, av.x, av.y);
                mma_16816<BF16>(acc[j], xv[0].z, xv[1].z, xv[0].w, xv[1].w, av.z, av.w);
            }
        };
        int k = ka;
#pragma unroll(NT >= 8 ? 2 : 4)
        for (; k + 32 <= kb; k += 32)
            step(true);
        if (k < kb) // the end of K: a multiple of 8
            step(k + t * 8 < kb);
        // each slot of the segment, ks-th slice
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = h * 8 + q;
            if (s >= s0 && s < s1) {
                float2 *to = reinterpret_cast<float2 *>(red) + ((ks * SB + s) * RB + 2 * t) / 2;
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    to[4 * j] = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < SB * (RB / 4); i += LORA_THREADS) {
        const int s = i / (RB / 4), r = i % (RB / 4) * 4;
        if (slot0 + s >= p.slots || r0 + r >= p.R)
            continue;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int ks = 0; ks < slices; ++ks) {
            const float4 v = red[((ks * SB + s) * RB + r) / 4];
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
        }
        // (slots without an adapter get whatever is there: never read back)
        *reinterpret_cast<float4 *>(p.v + ((size_t)blockIdx.z * p.slots + slot0 + s) * p.R + r0 + r) = sum;
    }
}

// ---------------------------------------------------------------- up

// A CTA's slots in the second kernel: segments (runs of one adapter), rows.
struct UpSlots {
    float scale[LORA_UP_SLOTS]; // of the slot's adapter
    int first[LORA_UP_SLOTS + 1], adapter[LORA_UP_SLOTS], row[LORA_UP_SLOTS];
};

// Segments of 8 slots from slot0 on; returns how many.
__device__ __forceinline__ int read_segments(const LoraParams &p, int slot0, UpSlots &u, int &adapter)
{
    constexpr int SB = LORA_UP_SLOTS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Slot mine = read_slot(p, lane < SB ? slot0 + lane : p.slots);
    const uint32_t starts = segment_starts(mine.adapter, lane, SB);
    const int segs = __popc(starts);
    if (warp == 0 && lane < SB) {
        if ((starts >> lane) & 1u) {
            const int i = __popc(starts & ((1u << lane) - 1u));
            u.first[i] = lane;
            u.adapter[i] = mine.adapter;
        }
        if (lane == 0)
            u.first[segs] = SB;
        u.row[lane] = mine.row;
    }
    __syncthreads();
    adapter = mine.adapter;
    return segs;
}

// v of the CTA's slots into part[slot][rank / 4] from the first kernel's k
// ranges.  Thread: one float4 of ranks of one slot, a share of the ranges if
// there are threads to spare; the shares are joined in order.
__device__ __forceinline__ void sum_ranges(const LoraParams &p, int slot0, float4 *part)
{
    const int tid = threadIdx.x;
    const int r4 = p.R / 4;
    const int items = min(LORA_UP_SLOTS, p.slots - slot0) * r4;
    const int shares = max(1, min(p.splits, LORA_THREADS / items));
    const int per = (p.splits + shares - 1) / shares;
    const long step = (long)p.slots * r4;
    const float4 *src = reinterpret_cast<const float4 *>(p.v) + (long)slot0 * r4;
    for (int i = tid; i < items * shares; i += LORA_THREADS) {
        const int item = i % items, z0 = i / items * per, z1 = min(z0 + per, p.splits);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int z = z0; z < z1; ++z) {
            const float4 v = __ldcg(src + z * step + item);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
        }
        part[i] = sum;
    }
    __syncthreads();
    if (shares > 1) {
        // (then there are at most LORA_THREADS items, one per thread)
        if (tid < items) {
            float4 sum = part[tid];
            for (int z = 1; z < shares; ++z) {
                const float4 v = part[z * items + tid];
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            part[tid] = sum;
        }
        __syncthreads();
    }
}

// Ranks up to 16: 8 slots and `p.n_chunk` columns per CTA.  A warp's job is 64 columns of one
// segment, two per lane, all ranks in FP32: with one or two rows per
// adapter, as in a decode batch, that takes a third of the instructions of an
// MMA with its 16 rows.
template <bool BF16>
__global__ void __launch_bounds__(LORA_THREADS, 4) lora_up_kernel(const LoraParams p)
{
    constexpr int SB = LORA_UP_SLOTS;
    extern __shared__ float4 part[]; // [share][slot][rank / 4]
    __shared__ UpSlots u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Everything but v is ready: the first kernel let this one start only
    // after its own wait for the kernels before it.  So the slots and the
    // first job's operands are read while the first kernel runs.
    const int slot0 = blockIdx.x * SB;
    int adapter;
    const int segs = read_segments(p, slot0, u, adapter);

    const int n_lo = blockIdx.y * p.n_chunk, n_hi = n_lo + min(p.n_chunk, p.N - n_lo);
    // the job's B: the 8 or 16 ranks of columns n and n + 1 (zero past R; a
    // column pair past the end reads the last one's and is not stored)
    uint4 b[2][2];
    auto load_b = [&](int g, int n) {
        const uint16_t *base = static_cast<const uint16_t *>(p.lora_b) + ((long)g * p.N + min(n, n_hi - 2)) * p.R;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[c][h] = 8 * h < p.R ? __ldg(reinterpret_cast<const uint4 *>(base + (long)c * p.R) + h)
                                      : make_uint4(0u, 0u, 0u, 0u);
    };
    uint32_t cv[SB];
    auto load_c = [&](int s0, int s1, int n) {
#pragma unroll
        for (int s = 0; s < SB; ++s)
            if (s >= s0 && s < s1 && n < n_hi)
                cv[s] = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.c) +
                                                            (long)u.row[s] * p.ld_c + n);
    };
    int seg = warp - LORA_WARPS, n0 = n_lo;
    auto advance = [&]() { // to this warp's next job
        seg += LORA_WARPS;
        while (seg >= segs) {
            seg -= segs;
            n0 += 64;
        }
    };
    auto load_job = [&]() {
        const int g = u.adapter[seg];
        if (g >= 0) {
            load_b(g, n0 + 2 * lane);
            load_c(u.first[seg], u.first[seg + 1], n0 + 2 * lane);
        }
    };
    advance();
    if (n0 < n_hi)
        load_job();
    if (warp == 0 && lane < SB) // read after the next barriers
        u.scale[lane] = adapter >= 0 ? __ldg(p.scales + adapter) : 0.0f;

    grid_dependency_wait();
    grid_launch_dependents();

    sum_ranges(p, slot0, part);
    const int r4 = p.R / 4;

    bool loaded = true;
    for (; n0 < n_hi; advance(), loaded = false) {
        const int g = u.adapter[seg];
        if (g < 0)
            continue;
        if (!loaded)
            load_job();
        const int s0 = u.first[seg], s1 = u.first[seg + 1];
        const int n = n0 + 2 * lane;
        float acc[SB][2];
#pragma unroll
        for (int s = 0; s < SB; ++s)
            acc[s][0] = acc[s][1] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float w[2][8];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t raw[4] = {b[c][h].x, b[c][h].y, b[c][h].z, b[c][h].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2<BF16>(raw[i]);
                    w[c][2 * i] = f.x;
                    w[c][2 * i + 1] = f.y;
                }
            }
            if (8 * h >= p.R) // past R: neither v nor B
                break;
#pragma unroll
            for (int s = 0; s < SB; ++s) {
                if (s < s0 || s >= s1)
                    continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 v = part[s * r4 + 2 * h + i];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        acc[s][c] = fmaf(v.x, w[c][4 * i], acc[s][c]);
                        acc[s][c] = fmaf(v.y, w[c][4 * i + 1], acc[s][c]);
                        acc[s][c] = fmaf(v.z, w[c][4 * i + 2], acc[s][c]);
                        acc[s][c] = fmaf(v.w, w[c][4 * i + 3], acc[s][c]);
                    }
                }
            }
        }
        if (n < n_hi) {
#pragma unroll
            for (int s = 0; s < SB; ++s) {
                if (s < s0 || s >= s1)
                    continue;
                const float2 old = unpack2<BF16>(cv[s]);
                const float f = u.scale[s];
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.d) + (long)u.row[s] * p.ld_d + n) =
                    pack2<BF16>(fmaf(f, acc[s][0], old.x), fmaf(f, acc[s][1], old.y));
            }
        }
    }
}

// Ranks above 16: the same cut, but a warp's job is 32 columns of one segment
// with mma.sync, v in two 16-bit terms (hi + lo: 16 bits of mantissa with BF16,
// 22 with FP16, so that the middle result costs no accuracy; an FP16 row is
// divided by a power of two first, so that v may exceed its range).  Rank 64,
// 64 rows of 28 adapters, N = 7168, K = 2048: in FP32 20.2 us a call, most of it
// reading B, whose columns a lane of that form has 2 R bytes from the next lane's;
// here four lanes read 64 bytes of a column: 15.9 us, where the weights take 5
// (256 rows: 38.1 -> 22.3).  Half of an MMA's rows are empty, and adapters that
// begin within 8 slots are read by both their blocks.  The MMA's columns are dealt out so that a lane's results
// are 8 columns side by side.
template <bool BF16>
__global__ void __launch_bounds__(LORA_THREADS, 3) lora_up_mma_kernel(const LoraParams p)
{
    constexpr int SB = LORA_UP_SLOTS;
    extern __shared__ float4 part[]; // [share][slot][rank / 4], then hi and lo [slot][rank]
    __shared__ UpSlots u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane & 3, q = lane >> 2; // q: slot, or column of B
    // (read early: see above)
    const int slot0 = blockIdx.x * SB;
    int adapter;
    const int segs = read_segments(p, slot0, u, adapter);

    const int n_lo = blockIdx.y * p.n_chunk, n_hi = n_lo + min(p.n_chunk, p.N - n_lo);
    int seg = warp - LORA_WARPS, n0 = n_lo;
    auto advance = [&]() { // to this warp's next job
        do {
            seg += LORA_WARPS;
            while (seg >= segs) {
                seg -= segs;
                n0 += 32;
            }
        } while (n0 < n_hi && u.adapter[seg] < 0);
    };
    // ranks k0 + 8 t to k0 + 8 t + 7 of columns n0 + 8 (q / 2) + q % 2 + 0, 2, 4, 6
    auto load_b = [&](uint4 (&b)[4], int k0) {
        const int n = n0 + 8 * (q >> 1) + (q & 1);
        const bool in = n < n_hi && k0 + 8 * t < p.R; // (N is a multiple of 8)
        const uint16_t *src = static_cast<const uint16_t *>(p.lora_b) + ((long)u.adapter[seg] * p.N + n) * p.R + k0 + 8 * t;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b[j] = in ? __ldg(reinterpret_cast<const uint4 *>(src + 2 * j * (long)p.R)) : make_uint4(0u, 0u, 0u, 0u);
    };
    // columns n0 + 8 t to n0 + 8 t + 7 of slot q
    auto mine = [&]() { return q >= u.first[seg] && q < u.first[seg + 1] && n0 + 8 * t < n_hi; };
    auto load_c = [&]() {
        return mine() ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.c) + (long)u.row[q] * p.ld_c +
                                                         n0 + 8 * t)
                      : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 b[4], c = make_uint4(0u, 0u, 0u, 0u);
    advance();
    if (n0 < n_hi) {
        load_b(b, 0);
        c = load_c();
    }
    if (warp == 0 && lane < SB) // read after the next barriers
        u.scale[lane] = adapter >= 0 ? __ldg(p.scales + adapter) : 0.0f;

    grid_dependency_wait();
    grid_launch_dependents();
    sum_ranges(p, slot0, part);

    // warp: the terms of one slot, with zeros up to a multiple of 32 ranks
    const int ranks = (p.R + 31) / 32 * 32, pitch = 2 * ranks + 64; // (bytes)
    const uint32_t hi_at = smem_addr(part) + (uint32_t)lora_up_part(p.R), lo_at = hi_at + (uint32_t)(SB * pitch);
    {
        const int r4 = p.R / 4;
        float amax = 0.0f, power = 1.0f;
        if constexpr (!BF16) {
            for (int i = lane; i < r4; i += 32) {
                const float4 v = part[warp * r4 + i];
                amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
            }
            power = lora_fp16_scale(amax);
        }
        const float inv = 1.0f / power; // a power of two: exact
        for (int i = lane; i < ranks / 4; i += 32) {
            const float4 v = i < r4 ? part[warp * r4 + i] : make_float4(0.f, 0.f, 0.f, 0.f);
            uint32_t hi[2], lo[2];
            split_two<BF16>(v.x * inv, v.y * inv, hi[0], lo[0]);
            split_two<BF16>(v.z * inv, v.w * inv, hi[1], lo[1]);
            const uint32_t at = (uint32_t)(warp * pitch + i * 8);
            st_shared_v2(hi_at + at, hi[0], hi[1]);
            st_shared_v2(lo_at + at, lo[0], lo[1]);
        }
        if (lane == 0)
            u.scale[warp] *= power;
    }
    __syncthreads();

    float acc[4][4] = {};
    for (int k0 = 0; n0 < n_hi;) {
        // what comes next is on its way while this is worked on
        uint16_t *to = static_cast<uint16_t *>(p.d) + (long)u.row[q] * p.ld_d + n0 + 8 * t;
        const bool store = mine(), last = k0 + 32 >= p.R;
        const uint32_t at = (uint32_t)(q * pitch + (k0 + 8 * t) * 2);
        uint4 next_b[4], next_c = c;
        k0 = last ? 0 : k0 + 32;
        if (last)
            advance();
        if (n0 < n_hi) {
            load_b(next_b, k0);
            if (last)
                next_c = load_c();
        }
#pragma unroll
        for (int term = 0; term < 2; ++term) {
            const uint4 v = ld_shared_v4((term ? lo_at : hi_at) + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma_16816<BF16>(acc[j], v.x, 0u, v.y, 0u, b[j].x, b[j].y);
                mma_16816<BF16>(acc[j], v.z, 0u, v.w, 0u, b[j].z, b[j].w);
            }
        }
        if (last) {
            if (store) {
                const uint32_t old[4] = {c.x, c.y, c.z, c.w};
                const float f = u.scale[q];
                uint32_t out[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 o = unpack2<BF16>(old[j]);
                    out[j] = pack2<BF16>(fmaf(f, acc[j][0], o.x), fmaf(f, acc[j][1], o.y));
                }
                st_global_v4(to, out[0], out[1], out[2], out[3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b[j] = next_b[j];
        c = next_c;
    }
}

// Overlapping the kernel before (`overlap`), except under a bound on the SMs,
// where two kernels at once would take more.
cudaError_t launch_one(void (*kernel)(LoraParams), dim3 grid, size_t smem, const LoraParams &p, bool overlap,
                       cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(LORA_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool BF16, int NT>
cudaError_t down(LoraParams p, bool overlap, int most_rank_blocks, cudaStream_t stream)
{
    const int rank_blocks = (p.R + 8 * NT - 1) / (8 * NT);
    cudaError_t err = cudaSuccess;
    for (p.rank_block = 0; err == cudaSuccess && p.rank_block < rank_blocks; p.rank_block += most_rank_blocks) {
        const int n = min(most_rank_blocks, rank_blocks - p.rank_block);
        const dim3 grid((unsigned)((p.slots + LORA_SLOTS - 1) / LORA_SLOTS), (unsigned)n, (unsigned)p.splits);
        err = launch_one(lora_down_kernel<BF16, NT>, grid, 0, p, overlap, stream);
    }
    return err;
}

template <bool BF16>
cudaError_t up(const LoraParams &p, bool overlap, cudaStream_t stream)
{
    const dim3 grid((unsigned)((p.slots + LORA_UP_SLOTS - 1) / LORA_UP_SLOTS),
                    (unsigned)(((long)p.N + p.n_chunk - 1) / p.n_chunk), 1);
    if (p.R <= LORA_FP32_RANK)
        return launch_one(lora_up_kernel<BF16>, grid, (size_t)lora_up_part(p.R), p, overlap, stream);
    const size_t terms = 2u * LORA_UP_SLOTS * (size_t)(2 * ((p.R + 31) / 32 * 32) + 64);
    return launch_one(lora_up_mma_kernel<BF16>, grid, (size_t)lora_up_part(p.R) + terms, p, overlap, stream);
}

template <bool BF16>
cudaError_t both(const LoraParams &p, bool overlap, int most_rank_blocks, cudaStream_t stream)
{
    const cudaError_t err = p.R <= 16 ? down<BF16, 2>(p, overlap, most_rank_blocks, stream)
                          : p.R <= 32 ? down<BF16, 4>(p, overlap, most_rank_blocks, stream)
                                      : down<BF16, 8>(p, overlap, most_rank_blocks, stream);
    if (err != cudaSuccess)
        return err;
    return up<BF16>(p, overlap, stream);
}

long slot_blocks(int slots, int size) { return slots > 0 ? ((long)slots + size - 1) / size : 1; }

// k in `splits` ranges, or a few less: multiples of 64, at least that.
void set_splits(LoraParams &p, long splits)
{
    const long most = min(((long)p.K + 63) / 64, 32L);
    splits = splits < 1 ? 1 : splits > most ? most : splits;
    p.k_chunk = (int)((p.K + splits * 64 - 1) / (splits * 64) * 64);
    p.splits = (int)(((long)p.K + p.k_chunk - 1) / p.k_chunk);
}

// N in `chunks` chunks, or a few less.
void set_columns(LoraParams &p, long chunks)
{
    const long chunk = ((long)p.N + chunks - 1) / chunks;
    p.n_chunk = (int)((chunk + 63) / 64 * 64);
}

// How a call is cut up, from its sizes alone (the workspace follows from it):
// k ranges and column chunks so that either kernel has about four CTAs per SM
// (three with mma.sync in the second: rank 64, 64 rows 15.9 us, 17.1 with four),
// at most 32 ranges (which the second kernel adds up in one or two rounds of
// loads), at least 64 wide.
void lora_plan(LoraParams &p)
{
    set_splits(p, 4 * 148 / (slot_blocks(p.slots, LORA_SLOTS) * ((p.R + 63) / 64)));
    const long up_ctas = (p.R <= LORA_FP32_RANK ? 4 : 3) * 148;
    const long chunk = ((long)p.N * slot_blocks(p.slots, LORA_UP_SLOTS) + up_ctas - 1) / up_ctas;
    p.n_chunk = (int)((min(chunk, (long)p.N) + 63) / 64 * 64);
}

// Under a bound on the SMs no launch has more CTAs than that: as many slots at a
// time as go into it, k and N cut so that the rest of the SMs have work too.
template <bool BF16>
cudaError_t launch_bounded(const LoraParams &all, int sms, cudaStream_t stream)
{
    const int rank_blocks = all.R <= 32 ? 1 : (all.R + 63) / 64;
    const int wide = rank_blocks > 2 ? rank_blocks : 2; // most CTAs of either kernel per block of 16 slots
    const int blocks = (int)min(slot_blocks(all.slots, LORA_SLOTS), (long)(sms / wide > 0 ? sms / wide : 1));
    const int step = sms > 1 ? blocks * LORA_SLOTS : LORA_UP_SLOTS;
    for (int first = 0; first < all.slots; first += step) {
        LoraParams p = lora_piece(all, first, min(step, all.slots - first));
        // (within the workspace of the call, which the pieces use in turn)
        const long room = (long)all.splits * all.slots / p.slots;
        set_splits(p, min((long)(sms / (blocks * rank_blocks)), room));
        set_columns(p, max(1L, sms / slot_blocks(p.slots, LORA_UP_SLOTS)));
        const cudaError_t err = both<BF16>(p, false, min(rank_blocks, sms), stream);
        if (err != cudaSuccess)
            return err;
    }
    return cudaSuccess;
}

} // namespace

long long lora_workspace(int slots, int R, int N, int K)
{
    LoraParams p = {};
    p.slots = slots;
    p.R = R;
    p.N = N;
    p.K = K;
    lora_plan(p);
    return (long long)p.splits * slots * R * 4;
}

cudaError_t launch_lora(const LoraParams &call, bool bf16, const DeviceView &dev, cudaStream_t stream)
{
    LoraParams p = call;
    lora_plan(p);
    if (dev.bounded)
        return bf16 ? launch_bounded<true>(p, dev.sms, stream) : launch_bounded<false>(p, dev.sms, stream);
    const int all = LORA_MAX_RANK; // blocks of ranks
    return bf16 ? both<true>(p, true, all, stream) : both<false>(p, true, all, stream);
}

} // namespace fp8nt
