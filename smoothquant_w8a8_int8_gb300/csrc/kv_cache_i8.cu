// Appending keys and values to a paged int8 cache, with the position rotation and the
// quantiser applied on the way.
//
// A rotated key or value row x of one token and head (kv_cache.cu has the rotation) is
// kept as symmetric codes and their scale,
//   scale = RN(max_d |x_d| / 127)  (1 where that is zero),
//   code_d = clamp(round_half_even(RN(x_d / scale)), +-127),
// so that it reads back as scale code_d, within scale / 2 of x_d.  The rotation's two
// products and their sum are rounded one by one here: a contraction would leave the
// codes to the compiler.  A row with an element that is not finite is kept as zeros
// with the scale NaN.
// Memory-bound like the append to a 16-bit cache: every projected element is read once
// and written once.  A head's row lies in D / 8 neighbouring threads' registers, its
// maximum is theirs by shuffles.
// Measured: 7976 tokens of 32 + 2 x 8 heads of 128 55 us, 348 MB at 94 % of the measured
// copy rate (codes by division in every place 73 us); 64 tokens 3.3 us, latency.
#include "kv_tokens.cuh"

#include <algorithm>

namespace sq {
namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ float max_or_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// (x, y) turned by the angle whose (cos, sin) are (c, s)
__device__ __forceinline__ void turn_pair(float &x, float &y, float c, float s) {
    const float x0 = x, y0 = y;
    x = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(y0, s));
    y = __fadd_rn(__fmul_rn(x0, s), __fmul_rn(y0, c));
}
// Four codes of a row, the first in the low byte, from the products with the scale's
// rounded reciprocal, and how far one is from its code at most.  A product p = RN(v RN(1
// / scale)) is within a relative 3 2^-24 of the quotient, |p| < 127.1, so both round to
// the same code unless p lies within 2^-14 of a half-integer.  Adding 1.5 2^23 rounds p
// to a whole number, half to even, whose low byte is the sum's.
__device__ __forceinline__ uint32_t near_codes(float4 x, float rscale, float &off) {
    const float magic = 12582912.0f;
    const unsigned long long r2 = pk(rscale, rscale), up = pk(magic, magic);
    const unsigned long long down = pk(-magic, -magic), minus = pk(-1.0f, -1.0f);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned long long p = mul2(i ? pk(x.z, x.w) : pk(x.x, x.y), r2);
        const unsigned long long k = add2(p, up);
        float a, b;
        upk(fma2(add2(k, down), minus, p), a, b);
        off = fmaxf(off, fmaxf(fabsf(a), fabsf(b)));
        upk(k, a, b);
        w[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
    }
    return __byte_perm(w[0], w[1], 0x5410);
}
// The same by divisions.
__device__ __noinline__ uint32_t exact_codes(float4 x, float scale) {
    const float v[4] = {x.x, x.y, x.z, x.w};
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i) {
        const float c = fminf(127.0f, fmaxf(-127.0f, rintf(__fdiv_rn(v[i], scale))));
        w |= (uint32_t)(__float2int_rn(c) & 0xff) << (8 * i);
    }
    return w;
}

// A row of blocks per token.  A unit is 8 elements of a head: for the "half" pairs
// elements 4u.. and rot/2 + 4u.., otherwise elements 8u...
__global__ void __launch_bounds__(kAppendThreads, 6) kv_append_i8_kernel(
    const float *QKV, int64_t T, int Hq, int Hkv, int D, const float *__restrict__ rope,
    int64_t rope_positions, int rot, int interleaved, const int *__restrict__ q_start,
    const int *__restrict__ kv_len, int B, const int *__restrict__ block_table,
    int64_t max_pages, int8_t *__restrict__ k_cache, int8_t *__restrict__ v_cache,
    float *__restrict__ k_scale, float *__restrict__ v_scale, int64_t num_pages, int page_shift,
    float *Qout, int64_t ldq) {
    pdl_launch_dependents();
    pdl_wait();
    const int heads = Hq + 2 * Hkv;
    const int upd_log = D == 128 ? 4 : 3, upd = 1 << upd_log;  // units per head: in one warp
    const int units = heads << upd_log;
    const int lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int b = token_sequence(q_start, B, (int)t, lane);
        if (b >= B || t < __ldg(q_start)) continue;  // no sequence's token
        const int64_t pos = (int64_t)__ldg(kv_len + b) - __ldg(q_start + b + 1) + t;
        const bool rotated = pos >= 0 && (rot == 0 || pos < rope_positions);
        int64_t page = -1;
        if (rotated && pos >> page_shift < max_pages)
            page = __ldg(block_table + b * max_pages + (pos >> page_shift));
        const bool stored = page >= 0 && page < num_pages;
        const float *src = QKV + t * heads * D;
        // whole warps go round, so that a head's maximum can be shuffled
        for (int u0 = blockIdx.y * kAppendThreads + threadIdx.x - lane; u0 < units;
             u0 += kAppendThreads * gridDim.y) {
            const int u = u0 + lane;
            const bool live = u < units;
            const int head = live ? u >> upd_log : 0, e = u & (upd - 1);
            const bool turn = head < Hq + Hkv && e < rot / 8;
            const bool split = turn && !interleaved;
            const int c0 = split ? 4 * e : 8 * e;              // the unit's first four elements
            const int c1 = split ? rot / 2 + 4 * e : 8 * e + 4;  // and its last four
            const float *x = src + head * D;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
            if (live) {
                a = *reinterpret_cast<const float4 *>(x + c0);
                d = *reinterpret_cast<const float4 *>(x + c1);
            }
            if (live && turn && rotated) {
                // (cos, sin) of pairs 4e .. 4e + 3
                const float4 *r = reinterpret_cast<const float4 *>(rope + pos * rot + 8 * e);
                const float4 r0 = __ldg(r), r1 = __ldg(r + 1);
                if (interleaved) {
                    turn_pair(a.x, a.y, r0.x, r0.y);
                    turn_pair(a.z, a.w, r0.z, r0.w);
                    turn_pair(d.x, d.y, r1.x, r1.y);
                    turn_pair(d.z, d.w, r1.z, r1.w);
                } else {
                    turn_pair(a.x, d.x, r0.x, r0.y);
                    turn_pair(a.y, d.y, r0.z, r0.w);
                    turn_pair(a.z, d.z, r1.x, r1.y);
                    turn_pair(a.w, d.w, r1.z, r1.w);
                }
            }
            float top = 0.0f;
            if (__any_sync(0xffffffffu, head >= Hq)) {
                top = max_or_nan(max_or_nan(max_or_nan(fabsf(a.x), fabsf(a.y)),
                                            max_or_nan(fabsf(a.z), fabsf(a.w))),
                                 max_or_nan(max_or_nan(fabsf(d.x), fabsf(d.y)),
                                            max_or_nan(fabsf(d.z), fabsf(d.w))));
                top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 4));
                if (D == 128) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, 8));
            }
            if (!live) continue;
            if (head < Hq) {
                if (!rotated) a = d = make_float4(0.f, 0.f, 0.f, 0.f);
                float *o = Qout + t * ldq + head * D;
                *reinterpret_cast<float4 *>(o + c0) = a;
                *reinterpret_cast<float4 *>(o + c1) = d;
            } else if (stored) {
                const int hk = head - Hq;
                const bool key = hk < Hkv;
                const int64_t row = ((page * Hkv + (key ? hk : hk - Hkv)) << page_shift) +
                                    (pos & ((1 << page_shift) - 1));
                float scale = __fdiv_rn(top, 127.0f);
                if (scale == 0.0f) scale = 1.0f;
                uint32_t w0 = 0, w1 = 0;
                if (top <= 3.402823466e38f) {
                    const float rscale = __frcp_rn(scale);
                    float off = 0.0f;
                    w0 = near_codes(a, rscale, off);
                    w1 = near_codes(d, rscale, off);
                    // (a reciprocal below 2^-100 may leave fp32's range)
                    if (off > 0.49993896484375f || scale < 0x1p-100f) {  // 0.5 - 2^-14
                        w0 = exact_codes(a, scale);
                        w1 = exact_codes(d, scale);
                    }
                } else {
                    scale = __int_as_float(0x7fffffff);
                }
                int8_t *o = (key ? k_cache : v_cache) + row * D;
                *reinterpret_cast<uint32_t *>(o + c0) = w0;
                *reinterpret_cast<uint32_t *>(o + c1) = w1;
                if (e == 0) (key ? k_scale : v_scale)[row] = scale;
            }
        }
    }
}

}  // namespace

sq_status launch_kv_append_i8(const float *QKV, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                              const float *rope, int64_t rope_positions, int64_t rot,
                              int interleaved, const int32_t *q_start, const int32_t *kv_len,
                              int64_t B, const int32_t *block_table, int64_t max_pages,
                              int8_t *k_cache, int8_t *v_cache, float *k_scale, float *v_scale,
                              int64_t num_pages, int64_t page_size, float *Q, int64_t ldq,
                              cudaStream_t st) {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    // a few tokens: a unit per thread; many: a block per token (see launch_kv_append)
    const int64_t units = (Hq + 2 * Hkv) * D / 8;
    const int64_t gy = T <= 2 * di.sms ? (units + kAppendThreads - 1) / kAppendThreads : 1;
    const int64_t grid = std::min<int64_t>(T, (int64_t)di.sms * 64);
    int page_shift = 4;
    while (1 << page_shift < page_size) ++page_shift;
    return launch_pdl(kv_append_i8_kernel, dim3((unsigned)grid, (unsigned)gy),
                      dim3(kAppendThreads), 0, st, 1, QKV, T, (int)Hq, (int)Hkv, (int)D, rope,
                      rope_positions, (int)rot, interleaved, q_start, kv_len, (int)B, block_table,
                      max_pages, k_cache, v_cache, k_scale, v_scale, num_pages, page_shift, Q, ldq);
}

}  // namespace sq
