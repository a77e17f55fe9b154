// Appending keys and values to a paged cache, with the position rotation
// applied on the way, and the rotation's table.
//
// Token i of sequence b stands at position p = kv_len[b] - q_len[b] + i (the
// lengths count the tokens being appended).  Its query and key heads are
// rotated in pairs (x, y) of their first `rot` elements by the angle
// p * inv_freq[j]:
//   x' = x cos - y sin,   y' = x sin + y cos,
// pairs (j, j + rot/2) or, interleaved, (2j, 2j + 1).  Queries leave in fp32;
// keys and values are rounded once, to the cache's 16-bit type, into row
// p % page_size of page block_table[b][p / page_size].
// Memory-bound: every projected element is read once and written once.  Measured:
// 7976 tokens of 32 / 8 heads of 128, bf16: 54 us, 6.8 TB/s, the measured copy
// rate; 64 tokens 5 us, latency.
#include "kv_tokens.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace sq {
namespace {

constexpr int kAppendThreads = 256;

// cos and sin of position * inv_freq[j], the angle in double: at position 10^6
// an fp32 angle is off by up to 0.03 rad.
__global__ void rope_table_kernel(const float *__restrict__ inv_freq, int64_t total, int half,
                                  float2 *__restrict__ table) {
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        double sn, cs;
        sincos((double)(i / half) * (double)inv_freq[i % half], &sn, &cs);
        table[i] = make_float2((float)cs, (float)sn);
    }
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if (BF) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&v);
    }
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}

// A row of blocks per token.  A unit is 8 elements of a head: for the "half" pairs
// elements 4u.. and rot/2 + 4u.., otherwise elements 8u...
template <bool BF>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(
    const float *QKV, int64_t T, int Hq, int Hkv, int D, const float *__restrict__ rope,
    int64_t rope_positions, int rot, int interleaved, const int *__restrict__ q_start,
    const int *__restrict__ kv_len, int B, const int *__restrict__ block_table,
    int64_t max_pages, uint16_t *__restrict__ k_cache, uint16_t *__restrict__ v_cache,
    int64_t num_pages, int page_size, float *Qout, int64_t ldq) {
    pdl_launch_dependents();
    pdl_wait();
    const int heads = Hq + 2 * Hkv;
    const int upd = D / 8;  // units per head
    const int lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int b = token_sequence(q_start, B, (int)t, lane);
        if (b >= B || t < __ldg(q_start)) continue;  // no sequence's token
        const int64_t pos = (int64_t)__ldg(kv_len + b) - __ldg(q_start + b + 1) + t;
        const bool rotated = pos >= 0 && (rot == 0 || pos < rope_positions);
        int64_t page = -1;
        if (rotated && pos / page_size < max_pages)
            page = __ldg(block_table + b * max_pages + pos / page_size);
        const bool stored = page >= 0 && page < num_pages;
        const float *src = QKV + t * heads * D;
        for (int u = blockIdx.y * kAppendThreads + threadIdx.x; u < heads * upd;
             u += kAppendThreads * gridDim.y) {
            const int head = u / upd, e = u % upd;
            const bool turn = head < Hq + Hkv && e < rot / 8;
            const bool split = turn && !interleaved;
            const int c0 = split ? 4 * e : 8 * e;              // the unit's first four elements
            const int c1 = split ? rot / 2 + 4 * e : 8 * e + 4;  // and its last four
            const float *x = src + head * D;
            float4 a = *reinterpret_cast<const float4 *>(x + c0);
            float4 d = *reinterpret_cast<const float4 *>(x + c1);
            if (turn && rotated) {
                // (cos, sin) of pairs 4e .. 4e + 3
                const float4 *r = reinterpret_cast<const float4 *>(rope + pos * rot + 8 * e);
                const float4 r0 = __ldg(r), r1 = __ldg(r + 1);
                if (interleaved) {
                    const float4 a0 = a, d0 = d;
                    a.x = a0.x * r0.x - a0.y * r0.y;
                    a.y = a0.x * r0.y + a0.y * r0.x;
                    a.z = a0.z * r0.z - a0.w * r0.w;
                    a.w = a0.z * r0.w + a0.w * r0.z;
                    d.x = d0.x * r1.x - d0.y * r1.y;
                    d.y = d0.x * r1.y + d0.y * r1.x;
                    d.z = d0.z * r1.z - d0.w * r1.w;
                    d.w = d0.z * r1.w + d0.w * r1.z;
                } else {
                    const float4 a0 = a, d0 = d;
                    a.x = a0.x * r0.x - d0.x * r0.y;
                    d.x = a0.x * r0.y + d0.x * r0.x;
                    a.y = a0.y * r0.z - d0.y * r0.w;
                    d.y = a0.y * r0.w + d0.y * r0.z;
                    a.z = a0.z * r1.x - d0.z * r1.y;
                    d.z = a0.z * r1.y + d0.z * r1.x;
                    a.w = a0.w * r1.z - d0.w * r1.w;
                    d.w = a0.w * r1.w + d0.w * r1.z;
                }
            }
            if (head < Hq) {
                if (!rotated) a = d = make_float4(0.f, 0.f, 0.f, 0.f);
                float *o = Qout + t * ldq + head * D;
                *reinterpret_cast<float4 *>(o + c0) = a;
                *reinterpret_cast<float4 *>(o + c1) = d;
            } else if (stored) {
                const int hk = head - Hq;
                uint16_t *o = (hk < Hkv ? k_cache : v_cache) +
                              ((page * Hkv + (hk < Hkv ? hk : hk - Hkv)) * page_size +
                               pos % page_size) * D;
                const uint2 w0 = make_uint2(pack16<BF>(a.x, a.y), pack16<BF>(a.z, a.w));
                const uint2 w1 = make_uint2(pack16<BF>(d.x, d.y), pack16<BF>(d.z, d.w));
                *reinterpret_cast<uint2 *>(o + c0) = w0;
                *reinterpret_cast<uint2 *>(o + c1) = w1;
            }
        }
    }
}

}  // namespace

sq_status launch_rope_table(const float *inv_freq, int64_t positions, int64_t rot, float *table,
                            cudaStream_t st) {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    const int64_t total = positions * (rot / 2);
    const int64_t grid = std::min<int64_t>((total + 255) / 256, (int64_t)di.sms * 16);
    return launch_pdl(rope_table_kernel, dim3((unsigned)grid), dim3(256), 0, st, 1, inv_freq,
                      total, (int)(rot / 2), reinterpret_cast<float2 *>(table));
}

sq_status launch_kv_append(const float *QKV, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                           const float *rope, int64_t rope_positions, int64_t rot,
                           int interleaved, const int32_t *q_start, const int32_t *kv_len,
                           int64_t B, const int32_t *block_table, int64_t max_pages,
                           void *k_cache, void *v_cache, int cache_type, int64_t num_pages,
                           int64_t page_size, float *Q, int64_t ldq, cudaStream_t st) {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    // a few tokens: a unit per thread; many: a block per token (32 / 8 heads of 128,
    // that layout alone, cold L2, launch included: 64 tokens 7.8 and 9.9 us, 256: 8.6
    // and 9.7, 512: 11.9 and 12.5, 1024: 16.7 and 16.0, 2048: 24.8 and 22.9)
    const int64_t units = (Hq + 2 * Hkv) * D / 8;
    const int64_t gy = T <= 2 * di.sms ? (units + kAppendThreads - 1) / kAppendThreads : 1;
    const int64_t grid = std::min<int64_t>(T, (int64_t)di.sms * 64);
    return launch_pdl(
        cache_type == SQ_CACHE_BF16 ? kv_append_kernel<true> : kv_append_kernel<false>,
        dim3((unsigned)grid, (unsigned)gy), dim3(kAppendThreads), 0, st, 1, QKV, T, (int)Hq,
        (int)Hkv, (int)D, rope, rope_positions, (int)rot, interleaved, q_start, kv_len, (int)B,
        block_table, max_pages, static_cast<uint16_t *>(k_cache),
        static_cast<uint16_t *>(v_cache), num_pages, (int)page_size, Q, ldq);
}

}  // namespace sq
