// Low-rank adapters of many requests beside a shared projection:
//
//   d[t, n] = c[t, n] + scale_g * sum_r v[t, r] B_g[n, r],   v[t, r] = sum_k x[t, k] A_g[r, k]
//
// for every slot i with adapter g = m_indices[i] and row t = order[i].  Slots
// sorted by adapter (as group_rows_by_index leaves them) share the reads of
// its weights.
//
// Both factors are thin, so the operator is bound by reading x, c and the
// adapters and writing d, not by its products; mma.sync with operands loaded
// straight from global memory into fragments keeps them off that path (a
// 16-byte load gives a lane 8 consecutive elements of the reduction, which
// any pairing of the MMA's k positions may use as long as both operands use
// the same one).  Two kernels, the second set up while the first runs:
//   down  v in FP32 for a range of k per CTA (`splits` ranges, written side by
//         side: summed in order by the second kernel, so no atomics)
//   up    sums the ranges, splits v into two 16-bit terms (hi + lo: 16 bits of
//         mantissa with BF16, 22 with FP16, so that the middle result costs no
//         accuracy; FP16 rows are scaled by a power of two first, so that v
//         may exceed its range) and adds the product to c, rounding once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "grouped.h"
#include "ptx.cuh"

namespace fp8nt {

namespace {

constexpr int LORA_THREADS = 256;
constexpr int LORA_WARPS = 8;

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

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (BF16)
        return pack_bf16x2(lo, hi);
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// A slot's row and adapter, -1 where it has none (or a bad one, flagged).
struct Slot {
    int row;
    int adapter;
};

__device__ __forceinline__ Slot read_slot(const LoraParams &p, int i)
{
    Slot s = {-1, -1};
    if (i < p.slots) {
        const int g = __ldg(p.m_indices + i);
        const int t = p.order ? __ldg(p.order + i) : i;
        if (g >= 0 && t >= 0) {
            if (g < p.adapters && t < p.rows) {
                s.row = t;
                s.adapter = g;
            } else {
                atomicOr(p.status, DEVERR_BAD_INDEX);
            }
        }
    }
    return s;
}

// Bit i: a segment (run of one adapter) begins at slot i of a warp's slots, one
// slot per lane of the lowest `n` lanes.
__device__ __forceinline__ uint32_t segment_starts(int adapter, int lane, int n)
{
    const int before = __shfl_up_sync(0xffffffffu, adapter, 1);
    return __ballot_sync(0xffffffffu, lane < n && (lane == 0 || adapter != before));
}

// ---------------------------------------------------------------- down

// MT blocks of 16 slots per warp job, NT blocks of 8 ranks, WR groups of
// 16 * MT slots per CTA; the CTA's 8 / WR warps of a group share its k range.
template <bool BF16, int MT, int NT, int WR>
__global__ void __launch_bounds__(LORA_THREADS) lora_down_kernel(const LoraParams p)
{
    constexpr int SB = 16 * MT;         // slots of a group
    constexpr int WK = LORA_WARPS / WR; // warps of a group
    constexpr int RB = 8 * NT;          // ranks of this CTA
    extern __shared__ float red[];      // [WR][WK][SB][RB]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = warp / WK, wk = warp % WK;
    const int t = lane & 3, q = lane >> 2;
    grid_dependency_wait();
    grid_launch_dependents();
    const int slot0 = (blockIdx.x * WR + wr) * SB;
    const int r0 = blockIdx.y * RB;
    const Slot mine = read_slot(p, lane < SB ? slot0 + lane : p.slots);
    uint32_t starts = segment_starts(mine.adapter, lane, SB);
    const int segs = __popc(starts);
    const int ks_count = max(1, WK / segs); // k slices per segment
    const int k_lo = blockIdx.z * p.k_chunk, k_hi = min(k_lo + p.k_chunk, p.K);
    const int k_step = ((k_hi - k_lo + ks_count - 1) / ks_count + 63) / 64 * 64;
    float *my_red = red + (size_t)wr * WK * SB * RB;

    for (int job = wk; job < segs * ks_count; job += WK) {
        const int seg = job / ks_count, ks = job % ks_count;
        uint32_t left = starts;
        for (int i = 0; i < seg; ++i)
            left &= left - 1;
        const int s0 = __ffs(left) - 1;
        left &= left - 1;
        const int s1 = left ? __ffs(left) - 1 : SB;
        const int g = __shfl_sync(0xffffffffu, mine.adapter, s0);
        if (g < 0)
            continue;
        const uint16_t *xrow[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = m * 16 + h * 8 + q;
                const int row = __shfl_sync(0xffffffffu, mine.row, s);
                xrow[m][h] = s >= s0 && s < s1 ? static_cast<const uint16_t *>(p.x) + (size_t)row * p.ld_x : nullptr;
            }
        const uint16_t *arow[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int r = r0 + 8 * j + q;
            arow[j] = r < p.R ? static_cast<const uint16_t *>(p.lora_a) + ((size_t)g * p.R + r) * p.K : nullptr;
        }
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[m][j][e] = 0.0f;
        const int ka = k_lo + ks * k_step, kb = min(ka + k_step, k_hi);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
        for (int k = ka; k < kb; k += 32) {
            const int at = k + t * 8;
            const bool in = at < kb;
            uint4 xv[MT][2], av[NT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xv[m][h] = in && xrow[m][h] ? __ldg(reinterpret_cast<const uint4 *>(xrow[m][h] + at)) : zero;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                av[j] = in && arow[j] ? __ldg(reinterpret_cast<const uint4 *>(arow[j] + at)) : zero;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    mma_16816<BF16>(acc[m][j], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, av[j].x, av[j].y);
                    mma_16816<BF16>(acc[m][j], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, av[j].z, av[j].w);
                }
        }
        // each row of the segment, ks-th slice
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = m * 16 + h * 8 + q;
                if (s >= s0 && s < s1) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        *reinterpret_cast<float2 *>(my_red + ((size_t)ks * SB + s) * RB + 8 * j + 2 * t) =
                            make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                }
            }
    }
    __syncthreads();
    // sum the slices; the group's warps share its slots
    const int gt = threadIdx.x - wr * WK * 32;
    for (int i = gt; i < SB * (RB / 4); i += WK * 32) {
        const int s = i / (RB / 4), r = i % (RB / 4) * 4;
        if (slot0 + s >= p.slots || r0 + r >= p.R)
            continue;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int ks = 0; ks < ks_count; ++ks) {
            const float4 v = *reinterpret_cast<const float4 *>(my_red + ((size_t)ks * SB + s) * RB + r);
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

// MT blocks of 16 slots per CTA (all its warps), `p.n_chunk` columns per CTA.
template <bool BF16, int MT>
__global__ void __launch_bounds__(LORA_THREADS) lora_up_kernel(const LoraParams p)
{
    constexpr int SB = 16 * MT;
    extern __shared__ uint8_t smem[];
    // v as two 16-bit terms, [SB][pitch] each; pitch: R rounded up to 16, plus
    // 8 so that the 8 rows of a fragment load fall into distinct banks
    const int pitch = (p.R + 15) / 16 * 16 + 8;
    uint16_t *hi = reinterpret_cast<uint16_t *>(smem);
    uint16_t *lo = hi + SB * pitch;
    __shared__ float row_scale[SB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane & 3, q = lane >> 2;
    grid_dependency_wait();
    grid_launch_dependents();
    const int slot0 = blockIdx.x * SB;
    const Slot mine = read_slot(p, lane < SB ? slot0 + lane : p.slots);
    const uint32_t starts = segment_starts(mine.adapter, lane, SB);
    const int segs = __popc(starts);

    // v of the CTA's slots: each warp sums the ranges of its rows in order
    for (int s = warp; s < SB; s += LORA_WARPS) {
        const int g = __shfl_sync(0xffffffffu, mine.adapter, s);
        if (g < 0)
            continue;
        const float *src = p.v + (size_t)(slot0 + s) * p.R;
        const size_t step = (size_t)p.slots * p.R;
        float scale = 1.0f;
        float keep[8]; // R <= 256: lane + 32 i
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = lane + 32 * i;
            float sum = 0.0f;
            if (r < p.R) {
#pragma unroll 8
                for (int z = 0; z < p.splits; ++z)
                    sum += __ldcg(src + z * step + r);
            }
            keep[i] = sum;
            amax = fmaxf(amax, fabsf(sum));
        }
        if constexpr (!BF16) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            // the largest value into [2^12, 2^13): both terms are normal
            // numbers down to 2^-15 of it
            if (amax > 0.0f && amax < __int_as_float(0x7f800000)) {
                const int e = min(max(ilogbf(amax) - 12, -100), 115);
                scale = ldexpf(1.0f, e);
            }
        }
        const float inv = 1.0f / scale; // a power of two: exact
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = lane + 32 * i;
            if (r < pitch - 8) {
                const float v = keep[i] * inv; // 0 past R
                const uint32_t h = pack2<BF16>(v, 0.0f);
                const float top = unpack2<BF16>(h).x;
                // an infinite or NaN v has no second term
                const float rest = isfinite(top) ? v - top : 0.0f;
                hi[s * pitch + r] = (uint16_t)h;
                lo[s * pitch + r] = (uint16_t)pack2<BF16>(rest, 0.0f);
            }
        }
        if (lane == 0)
            row_scale[s] = scale * __ldg(p.scales + g);
    }
    __syncthreads();

    // jobs: 32 columns of one segment
    const int n_lo = blockIdx.y * p.n_chunk, n_hi = min(n_lo + p.n_chunk, p.N);
    const int col_groups = (n_hi - n_lo + 31) / 32;
    for (int job = warp; job < segs * col_groups; job += LORA_WARPS) {
        const int seg = job % segs;
        uint32_t left = starts;
        for (int i = 0; i < seg; ++i)
            left &= left - 1;
        const int s0 = __ffs(left) - 1;
        left &= left - 1;
        const int s1 = left ? __ffs(left) - 1 : SB;
        const int g = __shfl_sync(0xffffffffu, mine.adapter, s0);
        if (g < 0)
            continue;
        const int n0 = n_lo + job / segs * 32;
        // MMA column c of block j is column n0 + (c / 2) * 8 + 2 j + c % 2, so
        // that a lane's results are 8 consecutive columns
        const uint16_t *brow[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + (q >> 1) * 8 + 2 * j + (q & 1);
            brow[j] = n < n_hi ? static_cast<const uint16_t *>(p.lora_b) + ((size_t)g * p.N + n) * p.R : nullptr;
        }
        const int col = n0 + t * 8;
        const bool col_ok = col < n_hi;
        float acc[MT][4][4];
        uint4 cv[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = m * 16 + h * 8 + q;
                const int row = __shfl_sync(0xffffffffu, mine.row, s);
                if (s >= s0 && s < s1 && col_ok)
                    cv[m][h] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.c) +
                                                                (size_t)row * p.ld_c + col);
            }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[m][j][e] = 0.0f;
#pragma unroll 2
        for (int k = 0; k < p.R; k += 16) {
            const int at = k + t * 4;
            uint2 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[j] = brow[j] && at < p.R ? __ldg(reinterpret_cast<const uint2 *>(brow[j] + at)) : make_uint2(0u, 0u);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m * 16 >= s1 || m * 16 + 16 <= s0)
                    continue;
                const uint16_t *h0 = hi + (m * 16 + q) * pitch + at, *l0 = lo + (m * 16 + q) * pitch + at;
                const uint2 ha = *reinterpret_cast<const uint2 *>(h0);
                const uint2 hb = *reinterpret_cast<const uint2 *>(h0 + 8 * pitch);
                const uint2 la = *reinterpret_cast<const uint2 *>(l0);
                const uint2 lb = *reinterpret_cast<const uint2 *>(l0 + 8 * pitch);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_16816<BF16>(acc[m][j], ha.x, hb.x, ha.y, hb.y, b[j].x, b[j].y);
                    mma_16816<BF16>(acc[m][j], la.x, lb.x, la.y, lb.y, b[j].x, b[j].y);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int s = m * 16 + h * 8 + q;
                const int row = __shfl_sync(0xffffffffu, mine.row, s);
                if (s >= s0 && s < s1 && col_ok) {
                    const float f = row_scale[s];
                    const uint32_t in[4] = {cv[m][h].x, cv[m][h].y, cv[m][h].z, cv[m][h].w};
                    uint32_t out[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 old = unpack2<BF16>(in[j]);
                        out[j] = pack2<BF16>(fmaf(f, acc[m][j][2 * h], old.x), fmaf(f, acc[m][j][2 * h + 1], old.y));
                    }
                    st_global_v4(static_cast<uint16_t *>(p.d) + (size_t)row * p.ld_d + col, out[0], out[1], out[2],
                                 out[3]);
                }
            }
    }
}

cudaError_t launch_pdl(void (*kernel)(LoraParams), dim3 grid, size_t smem, const LoraParams &p, cudaStream_t stream)
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool BF16, int MT, int NT, int WR>
cudaError_t down(const LoraParams &p, const LoraPlan &plan, cudaStream_t stream)
{
    constexpr size_t smem = sizeof(float) * LORA_WARPS * 16 * MT * 8 * NT;
    static std::atomic<bool> ready[64];
    auto kernel = lora_down_kernel<BF16, MT, NT, WR>;
    if (smem > 48 * 1024 && !ready[plan.device].load(std::memory_order_acquire)) {
        const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess)
            return err;
        ready[plan.device].store(true, std::memory_order_release);
    }
    const int slots_per_cta = 16 * MT * WR;
    const dim3 grid((unsigned)((p.slots + slots_per_cta - 1) / slots_per_cta), (unsigned)((p.R + 8 * NT - 1) / (8 * NT)),
                    (unsigned)p.splits);
    return launch_pdl(kernel, grid, smem, p, stream);
}

template <bool BF16, int MT, int WR>
cudaError_t down_rank(const LoraParams &p, const LoraPlan &plan, cudaStream_t stream)
{
    if (p.R <= 16)
        return down<BF16, MT, 2, WR>(p, plan, stream);
    if (p.R <= 32)
        return down<BF16, MT, 4, WR>(p, plan, stream);
    return down<BF16, MT, 8, WR>(p, plan, stream);
}

template <bool BF16, int MT>
cudaError_t up(const LoraParams &p, const LoraPlan &plan, cudaStream_t stream)
{
    const size_t smem = sizeof(uint16_t) * 2 * 16 * MT * ((p.R + 15) / 16 * 16 + 8);
    const dim3 grid((unsigned)((p.slots + 16 * MT - 1) / (16 * MT)), (unsigned)((p.N + p.n_chunk - 1) / p.n_chunk), 1);
    return launch_pdl(lora_up_kernel<BF16, MT>, grid, smem, p, stream);
}

template <bool BF16>
cudaError_t both(const LoraParams &p, const LoraPlan &plan, cudaStream_t stream)
{
    cudaError_t err = plan.wide ? down_rank<BF16, 2, 4>(p, plan, stream) : down_rank<BF16, 1, 1>(p, plan, stream);
    if (err != cudaSuccess)
        return err;
    return plan.wide ? up<BF16, 2>(p, plan, stream) : up<BF16, 1>(p, plan, stream);
}

} // namespace

// How a call is cut up, from its sizes alone (the workspace follows from it).
// Few slots: 16 per CTA and all 8 warps on one k range; many: 128 per CTA, 32
// per warp.  The k ranges and the column chunks are cut so that either kernel
// has about two CTAs per SM.
LoraPlan lora_plan(int slots, int R, int N, int K)
{
    LoraPlan plan = {};
    slots = slots > 0 ? slots : 1;
    plan.wide = slots > 256;
    const int sms = 148;
    const long down_blocks = (long)((slots + (plan.wide ? 127 : 15)) / (plan.wide ? 128 : 16)) *
                             ((R + 63) / 64);
    const int unit = plan.wide ? 128 : 256; // k of one pass of a CTA's warps
    long splits = (2 * sms + down_blocks - 1) / down_blocks;
    const long most = (K + unit - 1) / unit;
    splits = splits < 1 ? 1 : splits > most ? most : splits;
    plan.k_chunk = (int)((K + splits * unit - 1) / (splits * unit) * unit);
    plan.splits = (K + plan.k_chunk - 1) / plan.k_chunk;
    const long up_blocks = (slots + (plan.wide ? 31 : 15)) / (plan.wide ? 32 : 16);
    long chunks = (3 * sms + up_blocks - 1) / up_blocks;
    const long most_chunks = (N + 127) / 128;
    chunks = chunks < 1 ? 1 : chunks > most_chunks ? most_chunks : chunks;
    plan.n_chunk = (int)((N + chunks * 128 - 1) / (chunks * 128) * 128);
    return plan;
}

cudaError_t launch_lora(const LoraParams &p, const LoraPlan &plan, bool bf16, cudaStream_t stream)
{
    return bf16 ? both<true>(p, plan, stream) : both<false>(p, plan, stream);
}

} // namespace fp8nt
