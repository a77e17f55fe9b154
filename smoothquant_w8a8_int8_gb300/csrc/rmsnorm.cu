// Root-mean-square norm of a residual stream with the residual's addition and
// the next linear's activation quantiser fused in: the decoder's counterpart
// of the encoder's LayerNorm + quantiser.
//
// Per row m of H fp32 [M][K] (and residual R0, if given):
//   r_j = fl(H_j + R0_j)                  (stored to R when asked for)
//   ms  = fl(sum_j r_j^2 / K)             (fp32 sums in a tree)
//   y_j = fl(fl(r_j * rstd) * gamma_j),   rstd = RN(1 / sqrt(fl(ms + eps)))
// and the codes of y as the activation quantiser states them: v = fl(y / s),
// scale = fl(max|v| / 127) or the given one, code = round-half-even(fl(v / scale)).
// The row stays in registers from the one read of H and the residual to the
// codes: 8 bytes read and 4 + 2 written per element with the sum and the
// operand asked for.  Bound: memory and the codes' arithmetic together (54
// instructions an element: the definition's divisions, by reciprocals that are
// corrected or checked; 59 % of the issue slots).  Measured: 8192 x 4096 with
// sum and operand 85 us, 5.5 TB/s, 81 % of the measured copy rate; 1237 x 5136
// with a static scale 25 us; 16 x 4096 6.4 us, latency.
#include "decoder.cuh"
#include "row_codes.cuh"

#include <algorithm>
#include <mutex>

namespace sq {
namespace {

constexpr int kMaxRow = 16384;

// A group of tpr threads (whole warps) owns a row, VPT float4 of it in each
// thread's registers.  STATIC: the given scale; otherwise the row's own.  The
// smoothing factors, negated, and their reciprocals stand in shared-memory
// tables, or, for a block of one row (ONE), in registers: few rows are bound by
// latency, and a table costs them a round trip and a barrier.  The codes come
// from p = RN(RN(y RN(1/s)) RN(1/scale)) with the elements within 2^-14 of a
// half-integer on IEEE divisions: the same codes as the division's (p is within
// 4.2e-5 of fl(fl(y/s)/scale) for |quotient| <= 127.0001).  A row whose maximum
// is NaN or outside [2^-60, 2^100], and every row when a static scale lies
// outside [2^-60, 2^60] (fast == 0), takes IEEE divisions throughout.
template <bool STATIC, int VPT, bool ONE>
__global__ void __launch_bounds__(1024, 1) rmsnorm_quant_kernel(
    const float *H, const float *residual, const float *__restrict__ gamma, float eps,
    const float *__restrict__ s, int64_t rows, int K4, int tpr, float *R, float *Y,
    int8_t *__restrict__ q, float *__restrict__ scale, __nv_bfloat16 *__restrict__ op,
    int32_t *__restrict__ l1, float fixed_scale, int fast) {
    extern __shared__ float4 qtab[];
    float4 *nstab = qtab;      // -s
    float4 *ytab = qtab + K4;  // RN(1/s) or NaN
    __shared__ float red2[2][32];
    pdl_launch_dependents();
    pdl_wait();
    int rb = 0;  // the slot array of the group's next reduction (see row_group_reduce)
    const int rpb = blockDim.x / tpr;
    const int g = threadIdx.x / tpr;
    const int t = threadIdx.x % tpr;
    const float4 *s4 = reinterpret_cast<const float4 *>(s);
    const float4 *g4 = reinterpret_cast<const float4 *>(gamma);
    const int64_t tiles = (rows + rpb - 1) / rpb;
    // the row `ahead` tiles on into L2, while the next one is worked on
    auto prefetch = [&](int64_t tile) {
        const int64_t row = tile * rpb + g;
        if (ONE || t != 0 || tile >= tiles || row >= rows) return;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(H + row * K4 * 4),
                     "r"(K4 * 16)
                     : "memory");
        if (residual)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             residual + row * K4 * 4),
                         "r"(K4 * 16)
                         : "memory");
    };
    float4 ns_r[VPT], ys_r[VPT], g_r[VPT];  // (ONE)
    if (!ONE) {
        prefetch(blockIdx.x);
        for (int j = threadIdx.x; j < K4; j += blockDim.x) {
            const float4 v = __ldg(s4 + j);
            nstab[j] = make_float4(-v.x, -v.y, -v.z, -v.w);
            ytab[j] = make_float4(smooth_recip(v.x), smooth_recip(v.y), smooth_recip(v.z),
                                  smooth_recip(v.w));
        }
        __syncthreads();
    }
    const unsigned long long magic2 = pk(kRoundMagic, kRoundMagic);
    const float Kf = (float)(4 * K4);
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t row = tile * rpb + g;
        const bool valid = row < rows;
        const int64_t off = (valid ? row : 0) * K4;
        const float4 *h4 = reinterpret_cast<const float4 *>(H) + off;
        const float4 *r4 = reinterpret_cast<const float4 *>(residual) + off;
        float4 v[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = t + i * tpr;
            v[i] = (valid && j < K4) ? __ldcs(h4 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (ONE) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = t + i * tpr;
                ns_r[i] = j < K4 ? __ldg(s4 + j) : make_float4(1.f, 1.f, 1.f, 1.f);
                g_r[i] = j < K4 ? __ldg(g4 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        if (residual) {
            float4 r[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = t + i * tpr;
                r[i] = (valid && j < K4) ? __ldcs(r4 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            prefetch(tile + gridDim.x);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                v[i] = make_float4(v[i].x + r[i].x, v[i].y + r[i].y, v[i].z + r[i].z,
                                   v[i].w + r[i].w);
        } else {
            prefetch(tile + gridDim.x);
        }
        if (ONE) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const float4 x = ns_r[i];
                ys_r[i] = make_float4(smooth_recip(x.x), smooth_recip(x.y), smooth_recip(x.z),
                                      smooth_recip(x.w));
                ns_r[i] = make_float4(-x.x, -x.y, -x.z, -x.w);
            }
        }
        auto neg_s = [&](int i, int j) { return ONE ? ns_r[i] : nstab[j]; };
        auto recip_s = [&](int i, int j) { return ONE ? ys_r[i] : ytab[j]; };
        float sq = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = t + i * tpr;
            if (R && valid && j < K4) reinterpret_cast<float4 *>(R)[off + j] = v[i];
            sq += (v[i].x * v[i].x + v[i].y * v[i].y) + (v[i].z * v[i].z + v[i].w * v[i].w);
        }
        const float ms = __fdiv_rn(row_group_reduce<2>(sq, tpr, g, red2[rb]), Kf);
        rb ^= 1;
        // a row of zeros with eps = 0 is its own norm: zeros
        const float var = __fadd_rn(ms, eps);
        const float rstd = var == 0.0f ? 0.0f : __frsqrt_rn(var);
        // y (kept in v), and the row maximum of |fl(y / s)| by the corrected
        // reciprocal division on f32x2 pairs
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = t + i * tpr;
            if (j >= K4) continue;
            const float4 gv = ONE ? g_r[i] : __ldg(g4 + j);
            float4 y;
            y.x = __fmul_rn(__fmul_rn(v[i].x, rstd), gv.x);
            y.y = __fmul_rn(__fmul_rn(v[i].y, rstd), gv.y);
            y.z = __fmul_rn(__fmul_rn(v[i].z, rstd), gv.z);
            y.w = __fmul_rn(__fmul_rn(v[i].w, rstd), gv.w);
            if (Y && valid) reinterpret_cast<float4 *>(Y)[off + j] = y;
            v[i] = y;
            if (!STATIC) {
                const float4 ys = recip_s(i, j), ns = neg_s(i, j);
                const unsigned long long x01 = pk(y.x, y.y), x23 = pk(y.z, y.w);
                const unsigned long long y01 = pk(ys.x, ys.y), y23 = pk(ys.z, ys.w);
                const unsigned long long q01 = mul2(x01, y01), q23 = mul2(x23, y23);
                float d0, d1, d2, d3;
                upk(fma2(fma2(q01, pk(ns.x, ns.y), x01), y01, q01), d0, d1);
                upk(fma2(fma2(q23, pk(ns.z, ns.w), x23), y23, q23), d2, d3);
                m = max3_nan(m, max2_nan(fabsf(d0), fabsf(d1)), max2_nan(fabsf(d2), fabsf(d3)));
            }
        }
        bool exact = !fast;
        if (!STATIC) {
            m = row_group_reduce<0>(m, tpr, g, red2[rb]);
            rb ^= 1;
            exact = !(m >= 0x1p-60f && m <= 0x1p100f);
        }
        float sc = fixed_scale;
        if (!STATIC) {
            if (exact) {
                float me = 0.0f;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int j = t + i * tpr;
                    if (j >= K4) continue;
                    const float4 ns = neg_s(i, j);
                    me = fmaxf(me, fmaxf(abs_quotient(v[i].x, -ns.x), abs_quotient(v[i].y, -ns.y)));
                    me = fmaxf(me, fmaxf(abs_quotient(v[i].z, -ns.z), abs_quotient(v[i].w, -ns.w)));
                }
                m = row_group_reduce<1>(me, tpr, g, red2[rb]);
                rb ^= 1;
            }
            sc = m == 0.0f ? 1.0f : __fdiv_rn(m, 127.0f);
        }
        float a1 = 0.0f;
        if (valid) {
            if (t == 0) scale[row] = sc;
            const float rsc = __frcp_rn(sc);
            const unsigned long long r2 = pk(rsc, rsc);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = t + i * tpr;
                if (j >= K4) continue;
                const float4 ys = recip_s(i, j);
                const unsigned long long p01 = mul2(mul2(pk(v[i].x, v[i].y), pk(ys.x, ys.y)), r2);
                const unsigned long long p23 = mul2(mul2(pk(v[i].z, v[i].w), pk(ys.z, ys.w)), r2);
                const unsigned long long t01 = sub2(add2(p01, magic2), magic2);
                const unsigned long long t23 = sub2(add2(p23, magic2), magic2);
                float c[4], d[4];
                upk(t01, c[0], c[1]);
                upk(t23, c[2], c[3]);
                upk(sub2(p01, t01), d[0], d[1]);
                upk(sub2(p23, t23), d[2], d[3]);
                // NaN kept: a column whose s has no reciprocal
                const float dm = max3_nan(fabsf(d[0]), fabsf(d[1]),
                                          max2_nan(fabsf(d[2]), fabsf(d[3])));
                if (exact || !(dm <= kTieLimit)) {
                    const float4 ns = neg_s(i, j);
                    if (exact || !(fabsf(d[0]) <= kTieLimit)) c[0] = exact_code(v[i].x, -ns.x, sc);
                    if (exact || !(fabsf(d[1]) <= kTieLimit)) c[1] = exact_code(v[i].y, -ns.y, sc);
                    if (exact || !(fabsf(d[2]) <= kTieLimit)) c[2] = exact_code(v[i].z, -ns.z, sc);
                    if (exact || !(fabsf(d[3]) <= kTieLimit)) c[3] = exact_code(v[i].w, -ns.w, sc);
                }
                if (STATIC) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = fminf(127.0f, fmaxf(-127.0f, c[e]));
                }
                store4_codes(c[0], c[1], c[2], c[3], (off + j) * 4, q, op);
                a1 += (fabsf(c[0]) + fabsf(c[1])) + (fabsf(c[2]) + fabsf(c[3]));
            }
        }
        if (l1) {
            a1 = row_group_reduce<2>(a1, tpr, g, red2[rb]);  // exact: <= 127 * 16384 < 2^24
            rb ^= 1;
            if (valid && t == 0) l1[row] = (int32_t)a1;
        }
    }
}

using RmsKern = void (*)(const float *, const float *, const float *, float, const float *,
                         int64_t, int, int, float *, float *, int8_t *, float *,
                         __nv_bfloat16 *, int32_t *, float, int);

}  // namespace

sq_status launch_rmsnorm_quant(const float *H, const float *residual, const float *gamma,
                               float eps, const float *s, int64_t rows, int64_t K,
                               float static_scale, float *R, float *Y, int8_t *q, float *scale,
                               __nv_bfloat16 *op, int32_t *l1, cudaStream_t st) {
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    if (K > kMaxRow) return SQ_ERR_UNSUPPORTED;
    const int K4 = (int)(K / 4);
    // A block per row, its threads holding as few float4 as 1024 of them allow and
    // the column's factors in registers, while all rows are on the GPU at once; else
    // four float4 a thread and the factors in shared memory, and several rows per
    // block.  Measured, block per row against the other: 16 x 4096 8.7 and 11.8 us,
    // 152 x 4096 9.8 and 13.9, 304 x 4096 15.9 and 14.6, 152 x 8192 11.9 and 14.7,
    // 608 x 1024 8.8 and 9.9, 608 x 4096 24.2 and 16.1 (cold L2, launch included).
    const int vpt1 = K4 <= 1024 ? 1 : 2;
    const int tpr1 = ((K4 + vpt1 - 1) / vpt1 + 31) / 32 * 32;
    const bool one = K4 <= 2048 && rows <= (int64_t)di.sms * (1024 / tpr1);
    const int vpt = one ? vpt1 : 4;
    const int tpr = one ? tpr1 : ((K4 + 3) / 4 + 31) / 32 * 32;
    const int nt = one ? tpr : tpr * std::max(1, 256 / tpr);
    static const RmsKern kerns[2][3] = {
        {rmsnorm_quant_kernel<false, 1, true>, rmsnorm_quant_kernel<false, 2, true>,
         rmsnorm_quant_kernel<false, 4, false>},
        {rmsnorm_quant_kernel<true, 1, true>, rmsnorm_quant_kernel<true, 2, true>,
         rmsnorm_quant_kernel<true, 4, false>}};
    const int ki = static_scale > 0.0f ? 1 : 0, vi = one ? vpt - 1 : 2;
    const RmsKern kern = kerns[ki][vi];
    // the range of scales for which the product decides the code (see the kernel)
    const int fast = static_scale >= 0x1p-60f && static_scale <= 0x1p60f;
    const int smem = one ? 0 : K4 * 32;
    const int64_t tiles = (rows + nt / tpr - 1) / (nt / tpr);
    int64_t grid = tiles;
    if (!one) {
        static std::mutex mu;
        static bool opted[64][2] = {};
        std::lock_guard<std::mutex> lock(mu);
        bool &o = opted[di.device & 63][ki];
        if (!o) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kMaxRow * 8) != cudaSuccess)
                return SQ_ERR_CUDA;
            o = true;
        }
        // 64 registers a thread: 1024 threads per SM; as many blocks as fit at once
        grid = std::min<int64_t>(tiles, (int64_t)di.sms * std::max(1, 1024 / nt));
    }
    return launch_pdl(kern, dim3((unsigned)grid), dim3((unsigned)nt), (size_t)smem, st, 1, H,
                      residual, gamma, eps, s, rows, K4, tpr, R, Y, q, scale, op, l1,
                      static_scale, fast);
}

}  // namespace sq
