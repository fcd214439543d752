// Rows sorted by the group each belongs to: a stable counting sort whose
// results are the layout of the grouped products.
//
//   offsets[g + 1] = offsets[g] + ceil(rows of g / alignment) * alignment
//   slot(r) = offsets[g] + number of rows r' < r with the same group g
//
// Bound by latency: 5.0 us a call for 512 rows, 8.0 us for 262144 rows of 64
// groups, whose arrays (5 MB) are read and written in 0.8 (of 512 groups 15 us, of
// 1024 46: every CTA adds up the counts of all chunks).  A short call is
// done by one CTA in one launch.  Beyond that the rows are cut into contiguous
// chunks: one kernel counts each chunk's rows per group, a second one adds up
// the counts of the chunks before its own and places its rows.  No atomics on
// results: they do not depend on timing.
// Within a chunk every warp takes a contiguous run of rows, 32 at a time: a
// row's rank among its 32 is the number of lower lanes with the same group
// (match), so the order of equal rows is kept.
#include <cuda_runtime.h>

#include <atomic>
#include <stdint.h>

#include "grouped.h"
#include "ptx.cuh"

namespace fp8nt {

namespace {

constexpr int GROUP_THREADS = 512;
constexpr int GROUP_WARPS = GROUP_THREADS / 32;
constexpr int GROUP_BATCH = 8; // rows per lane whose groups are read at once

struct GroupArgs {
    const void *index;
    int *offsets;
    int *order;
    int *slots;
    int *m_indices;
    int *counts; // [chunks][groups] (more than one chunk)
    unsigned int *status;
    int rows;
    int groups;
    int alignment;
    int capacity;
    int chunk; // rows per chunk, a multiple of GROUP_THREADS
    int chunks;
};

// The group of row r, or -1 if it has none; `bad` collects values that are
// neither a group nor -1.
template <bool I64>
__device__ __forceinline__ int group_of(const GroupArgs &a, int r, bool &bad)
{
    if (I64) {
        const long long v = __ldg(static_cast<const long long *>(a.index) + r);
        if (v >= 0 && v < a.groups)
            return (int)v;
        bad |= v != -1;
    } else {
        const int v = __ldg(static_cast<const int *>(a.index) + r);
        if (v >= 0 && v < a.groups)
            return v;
        bad |= v != -1;
    }
    return -1;
}

// Per-warp counts of the chunk's rows in hist[warp][group].
template <bool I64>
__device__ __forceinline__ void count_chunk(const GroupArgs &a, int r0, int r1, int *hist, bool &bad)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < GROUP_WARPS * a.groups; i += GROUP_THREADS)
        hist[i] = 0;
    __syncthreads();
    const int per = a.chunk / GROUP_WARPS;
    const int w0 = r0 + warp * per, w1 = min(w0 + per, r1);
    int *mine = hist + warp * a.groups;
    for (int base = w0; base < w1; base += 32 * GROUP_BATCH) {
        int g[GROUP_BATCH];
#pragma unroll
        for (int i = 0; i < GROUP_BATCH; ++i) {
            const int r = base + 32 * i + lane;
            g[i] = r < w1 ? group_of<I64>(a, r, bad) : -1;
        }
#pragma unroll
        for (int i = 0; i < GROUP_BATCH; ++i)
            if (g[i] >= 0)
                atomicAdd(mine + g[i], 1);
    }
    __syncthreads();
}

template <bool I64>
__global__ void __launch_bounds__(GROUP_THREADS) group_count_kernel(const GroupArgs a)
{
    extern __shared__ int hist[];
    grid_dependency_wait();
    grid_launch_dependents();
    bool bad = false;
    const int r0 = blockIdx.x * a.chunk, r1 = min(r0 + a.chunk, a.rows);
    count_chunk<I64>(a, r0, r1, hist, bad);
    for (int g = threadIdx.x; g < a.groups; g += GROUP_THREADS) {
        int n = 0;
        for (int w = 0; w < GROUP_WARPS; ++w)
            n += hist[w * a.groups + g];
        a.counts[(size_t)blockIdx.x * a.groups + g] = n;
    }
}

template <bool I64>
__global__ void __launch_bounds__(GROUP_THREADS) group_place_kernel(const GroupArgs a)
{
    extern __shared__ int smem[];
    int *hist = smem;                             // [GROUP_WARPS][groups]: counts, then next slots
    int *total = smem + GROUP_WARPS * a.groups;   // [groups] rows of the group
    int *start = total + a.groups;                // [groups + 1] offsets
    __shared__ int part[GROUP_WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.groups;
    if (a.chunks == 1) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    bool bad = false;
    const int r0 = blockIdx.x * a.chunk, r1 = min(r0 + a.chunk, a.rows);
    // (with several chunks the counting kernel let this one start once every
    // one of its CTAs had passed its own wait: the index is there)
    count_chunk<I64>(a, r0, r1, hist, bad);
    if (bad)
        atomicOr(a.status, DEVERR_BAD_INDEX);
    if (a.chunks > 1) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    // rows of each group in all chunks, and in those before this one (in
    // start[] until the scan)
    if (a.chunks == 1) {
        for (int g = tid; g < G; g += GROUP_THREADS) {
            int all = 0;
#pragma unroll
            for (int w = 0; w < GROUP_WARPS; ++w)
                all += hist[w * G + g];
            total[g] = all;
            start[g] = 0;
        }
    } else {
        // all threads share the sums of a group: `parts` runs of chunks each
        const int parts = max(1, GROUP_THREADS / G), per = (a.chunks + parts - 1) / parts;
        for (int g = tid; g < G; g += GROUP_THREADS)
            total[g] = start[g] = 0;
        __syncthreads();
        for (int i = tid; i < G * parts; i += GROUP_THREADS) {
            const int g = i % G, c0 = i / G * per, c1 = min(c0 + per, a.chunks);
            int all = 0, before = 0;
#pragma unroll 8
            for (int c = c0; c < c1; ++c) {
                const int n = __ldcg(a.counts + (size_t)c * G + g);
                all += n;
                before += c < (int)blockIdx.x ? n : 0;
            }
            atomicAdd(total + g, all); // whole numbers: any order gives the same
            atomicAdd(start + g, before);
        }
    }
    __syncthreads();
    // exclusive scan of the padded totals; thread t owns `per` groups
    const int per = (G + GROUP_THREADS - 1) / GROUP_THREADS;
    const int g0 = min(tid * per, G), g1 = min(g0 + per, G);
    int mine = 0;
    for (int g = g0; g < g1; ++g)
        mine += (total[g] + a.alignment - 1) / a.alignment * a.alignment;
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d)
            incl += v;
    }
    if (lane == 31)
        part[warp] = incl;
    __syncthreads();
    int at = incl - mine;
#pragma unroll
    for (int w = 0; w < GROUP_WARPS; ++w)
        at += w < warp ? part[w] : 0;
    for (int g = g0; g < g1; ++g) {
        // the next free slot of every warp's rows of group g
        int n[GROUP_WARPS];
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w)
            n[w] = hist[w * G + g];
        int next = at + start[g];
#pragma unroll
        for (int w = 0; w < GROUP_WARPS; ++w) {
            hist[w * G + g] = next;
            next += n[w];
        }
        start[g] = at;
        if (blockIdx.x == 0)
            a.offsets[g] = at;
        at += (total[g] + a.alignment - 1) / a.alignment * a.alignment;
    }
    if (tid == GROUP_THREADS - 1) { // its groups are the last ones, or none
        start[G] = at;
        if (blockIdx.x == 0)
            a.offsets[G] = at;
    }
    __syncthreads();
    // place this chunk's rows
    {
        const int per_warp = a.chunk / GROUP_WARPS;
        const int w0 = r0 + warp * per_warp, w1 = min(w0 + per_warp, r1);
        int *next = hist + warp * G;
        bool ignore = false;
        for (int base = w0; base < w1; base += 32 * GROUP_BATCH) {
            int g[GROUP_BATCH];
#pragma unroll
            for (int i = 0; i < GROUP_BATCH; ++i) {
                const int r = base + 32 * i + lane;
                g[i] = r < w1 ? group_of<I64>(a, r, ignore) : -1;
            }
#pragma unroll
            for (int i = 0; i < GROUP_BATCH; ++i) {
                if (base + 32 * i >= w1)
                    break;
                const int r = base + 32 * i + lane;
                const uint32_t same = __match_any_sync(0xffffffffu, g[i]);
                int slot = -1;
                if (g[i] >= 0) {
                    slot = next[g[i]] + __popc(same & ((1u << lane) - 1u));
                    a.order[slot] = r;
                    if (a.m_indices)
                        a.m_indices[slot] = g[i];
                }
                if (a.slots && r < w1)
                    a.slots[r] = slot;
                __syncwarp();
                if (g[i] >= 0 && lane == 31 - __clz(same)) // the last of its group
                    next[g[i]] = slot + 1;
                __syncwarp();
            }
        }
    }
    // slots that hold no row: the padding of each group (groups dealt out to
    // the chunks) and everything behind the last segment
    for (int g = blockIdx.x * GROUP_WARPS + warp; g < G; g += a.chunks * GROUP_WARPS)
        for (int s = start[g] + total[g] + lane; s < start[g + 1]; s += 32) {
            a.order[s] = -1;
            if (a.m_indices)
                a.m_indices[s] = -1;
        }
    for (int s = start[G] + blockIdx.x * GROUP_THREADS + tid; s < a.capacity; s += a.chunks * GROUP_THREADS) {
        a.order[s] = -1;
        if (a.m_indices)
            a.m_indices[s] = -1;
    }
}

template <bool I64>
cudaError_t launch(const GroupArgs &a, int device, bool bounded, cudaStream_t stream)
{
    const size_t count_smem = sizeof(int) * (size_t)GROUP_WARPS * a.groups;
    const size_t place_smem = count_smem + sizeof(int) * (2u * (size_t)a.groups + 1u);
    static std::atomic<bool> ready[64];
    if (device < 0 || device >= 64)
        return cudaErrorInvalidDevice;
    if (!ready[device].load(std::memory_order_acquire)) {
        const int most = (int)sizeof(int) * ((GROUP_WARPS + 2) * RAGGED_MAX_GROUPS + 1);
        cudaError_t err =
            cudaFuncSetAttribute(group_count_kernel<I64>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (err == cudaSuccess)
            err = cudaFuncSetAttribute(group_place_kernel<I64>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (err != cudaSuccess)
            return err;
        ready[device].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.chunks, 1, 1);
    cfg.blockDim = dim3(GROUP_THREADS, 1, 1);
    cfg.dynamicSmemBytes = count_smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = bounded ? 0 : 1; // (two kernels at once would take twice the SMs of one)
    if (a.chunks > 1) {
        const cudaError_t err = cudaLaunchKernelEx(&cfg, group_count_kernel<I64>, a);
        if (err != cudaSuccess)
            return err;
    }
    cfg.dynamicSmemBytes = place_smem;
    return cudaLaunchKernelEx(&cfg, group_place_kernel<I64>, a);
}

} // namespace

// Rows per chunk, a multiple of GROUP_THREADS: up to 2048 rows in one chunk
// (one launch), else chunks of 2048, growing so that every CTA adds up the
// counts of at most GROUP_MAX_CHUNKS chunks, or of as many as there may be CTAs.
int group_rows_chunk(int rows, int max_chunks)
{
    const int unit = 4 * GROUP_THREADS;
    int chunk = rows <= unit ? rows : (int)(((long)rows + max_chunks - 1) / max_chunks);
    if (rows > unit && chunk < unit)
        chunk = unit;
    chunk = (chunk + GROUP_THREADS - 1) / GROUP_THREADS * GROUP_THREADS;
    return chunk > 0 ? chunk : GROUP_THREADS;
}

cudaError_t launch_group_rows(const void *index, bool i64, int rows, int groups, int alignment, int capacity,
                              int *offsets, int *order, int *slots, int *m_indices, int *counts,
                              const DeviceView &dev, cudaStream_t stream)
{
    GroupArgs a;
    a.index = index;
    a.offsets = offsets;
    a.order = order;
    a.slots = slots;
    a.m_indices = m_indices;
    a.counts = counts;
    a.status = dev.status;
    a.rows = rows;
    a.groups = groups;
    a.alignment = alignment;
    a.capacity = capacity;
    a.chunk = group_rows_chunk(rows, dev.bounded && dev.sms < GROUP_MAX_CHUNKS ? dev.sms : GROUP_MAX_CHUNKS);
    a.chunks = rows > 0 ? (rows + a.chunk - 1) / a.chunk : 1;
    return i64 ? launch<true>(a, dev.index, dev.bounded, stream) : launch<false>(a, dev.index, dev.bounded, stream);
}

} // namespace fp8nt
