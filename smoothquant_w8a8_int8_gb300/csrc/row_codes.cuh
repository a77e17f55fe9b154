// Row reductions, correctly rounded reciprocals and code stores shared by the
// activation quantisers, LayerNorm and the RMS norm (sm_103a device code).
#pragma once
#include "common.cuh"

namespace sq {
namespace {

constexpr float kRoundMagic = 12582912.0f;      // 1.5 * 2^23
constexpr float kTieLimit = 0.49993896484375f;  // 0.5 - 2^-14

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max2_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// RN(1/s) where the corrected reciprocal division is proven (|s| in
// [2^-20, 2^20]), NaN elsewhere: the division tables' entry for s
__device__ __forceinline__ float smooth_recip(float x) {
    const float a = fabsf(x);
    return (a >= 0x1p-20f && a <= 0x1p20f) ? __frcp_rn(x) : __int_as_float(0x7fffffff);
}

// Reductions across the tpr threads of row group g for the register and
// LayerNorm kernels, synchronised on the group's own named barrier (1 + g, tpr threads)
// instead of the block's, so that the groups of a block run their tiles
// independently.  The caller alternates two slot arrays between consecutive
// reductions: a slot is rewritten only after the group has passed the next
// reduction's barrier, hence after every thread read it, so one barrier per
// reduction is enough.
__device__ __forceinline__ void row_group_sync(int g, int tpr) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(tpr) : "memory");
}
template <int OP>  // 0: max (NaN kept), 1: max, 2: sum
__device__ __forceinline__ float row_group_reduce(float v, int tpr, int g, float *red) {
    auto op = [](float a, float b) {
        return OP == 0 ? max2_nan(a, b) : OP == 1 ? fmaxf(a, b) : a + b;
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr > 32) {
        const int wpg = tpr >> 5;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        row_group_sync(g, tpr);
        v = red[g * wpg];
        for (int w = 1; w < wpg; ++w) v = op(v, red[g * wpg + w]);
    }
    return v;
}

// Four codes (integer-valued floats) to the outputs at element offset off
// (a multiple of 4): bf16 operand (8 bytes) and/or int8 (4 bytes).
__device__ __forceinline__ void store4_codes(float t0, float t1, float t2, float t3, int64_t off,
                                             int8_t *q, __nv_bfloat16 *op) {
    if (op) {
        // integers |t| <= 127: the high half of the fp32 pattern is the exact bf16
        const uint2 w = make_uint2(__byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x7632),
                                   __byte_perm(__float_as_uint(t2), __float_as_uint(t3), 0x7632));
        *reinterpret_cast<uint2 *>(op + off) = w;
    }
    if (q) {
        // t + 1.5 * 2^23 holds the code in its low byte (two's complement)
        float f0, f1, f2, f3;
        upk(add2(pk(t0, t1), pk(kRoundMagic, kRoundMagic)), f0, f1);
        upk(add2(pk(t2, t3), pk(kRoundMagic, kRoundMagic)), f2, f3);
        *reinterpret_cast<uint32_t *>(q + off) =
            __byte_perm(__byte_perm(__float_as_uint(f0), __float_as_uint(f1), 0x0040),
                        __byte_perm(__float_as_uint(f2), __float_as_uint(f3), 0x0040), 0x5410);
    }
}

// The code of x as the definition states it: round_half_even(fl(fl(x / s) /
// scale)), clamped (IEEE divisions; the rare near-tie elements).  By value and
// not inlined, so that the caller's register arrays stay in registers.
__device__ __noinline__ float exact_code(float x, float s, float scale) {
    return fminf(127.0f, fmaxf(-127.0f, rintf(__fdiv_rn(__fdiv_rn(x, s), scale))));
}

// |fl(x / s)| (IEEE division), out of line for the rare exact path
__device__ __noinline__ float abs_quotient(float x, float s) { return fabsf(__fdiv_rn(x, s)); }

}  // namespace
}  // namespace sq
