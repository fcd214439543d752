// What the two forms of the low-rank adapters share: slots and 16-bit pairs.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "grouped.h"
#include "ptx.cuh"

namespace fp8nt {

// Two FP32 values rounded to nearest even in the operands' 16-bit type.
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

__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// v as hi + lo, two 16-bit terms, for two values; an infinite or NaN v has no
// second one.
template <bool BF16>
__device__ __forceinline__ void split_two(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack2<BF16>(a, b);
    const float2 top = unpack2<BF16>(hi);
    lo = pack2<BF16>(isfinite(top.x) ? a - top.x : 0.0f, isfinite(top.y) ? b - top.y : 0.0f);
}

// FP16 rows: the power of two that v is divided by, so that the largest of the
// warp's `amax` lands in [2^12, 2^13): both terms are then normal numbers for
// values down to 2^-15 of it.
__device__ __forceinline__ float lora_fp16_scale(float amax)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    if (amax > 0.0f && amax < __int_as_float(0x7f800000))
        return ldexpf(1.0f, min(max(ilogbf(amax) - 12, -100), 115));
    return 1.0f;
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
        if (g != -1 && t != -1) {
            if (g >= 0 && g < p.adapters && t >= 0 && t < p.rows) {
                s.row = t;
                s.adapter = g;
            } else {
                atomicOr(p.status, DEVERR_BAD_INDEX);
            }
        }
    }
    return s;
}

} // namespace fp8nt
