// Shared parts of the attention kernels over the paged cache: bounded waits,
// the CTA's share of the work, and the rows' last step.
#pragma once
#include "common.cuh"
#include "paged_line.cuh"

#include <cuda.h>
#include <cuda_fp16.h>

namespace sq {

namespace {

constexpr unsigned long long kPagedTimeoutNs = 4000000000ull;

__device__ __forceinline__ uint32_t su32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t gtime() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void bar_init(uint64_t *bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(bar)), "r"(count));
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort,
                                       unsigned *error) {
    const uint64_t t0 = gtime();
    for (uint32_t it = 1;; ++it) {
        if (try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort) return false;
            if (gtime() - t0 > kPagedTimeoutNs) {
                *abort = 1;
                atomicOr(error, 1u);
                return false;
            }
        }
    }
}
// Bounded wait for the phase of parity `parity`; false when the CTA aborted.
__device__ __forceinline__ bool wait_bar(const uint64_t *bar, uint32_t parity,
                                         volatile int *abort, unsigned *error) {
    const uint32_t a = su32(bar);
    if (try_wait(a, parity)) return true;
    return wait_slow(a, parity, abort, error);
}
// Every lane waits (so that every lane sees what the barrier publishes); the
// outcome is the warp's.
__device__ __forceinline__ bool warp_wait(const uint64_t *bar, uint32_t parity,
                                          volatile int *abort, unsigned *error) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, error)) != 0;
}
__device__ __forceinline__ void drain_bar(const uint64_t *bar, uint32_t parity,
                                          unsigned *error) {
    const uint32_t a = su32(bar);
    const uint64_t t0 = gtime();
    while (!try_wait(a, parity))
        if (gtime() - t0 > kPagedTimeoutNs) {
            atomicOr(error, 2u);
            return;
        }
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(bar)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(bar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                        int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(su32(bar)), "r"(x), "r"(y)
        : "memory");
}
// 2^x, relative error below 2^-22, results below 2^-126 flushed to zero
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(a - b) of two row maxima, 0 for a row maximum of no keys
__device__ __forceinline__ float max_factor(float a, float b) {
    return a == -INFINITY ? 0.0f : ex2(a - b);
}

// (a, b) as a pair of the cache's 16-bit type, a in the low half, and what the
// rounding left of each, rounded the same way: hi + lo is within 2^-18 (bf16)
// or 2^-22 (fp16) of the value, relative.
template <bool BF>
__device__ __forceinline__ void split16(float a, float b, uint32_t &hi, uint32_t &lo) {
    if (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        const __nv_bfloat162 l =
            __floats2bfloat162_rn(a - __low2float(h), b - __high2float(h));
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        const __half2 l = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}

// The line's length and this CTA's share of it, by all NT threads of the
// block: each sums a run of sequences, a scan over the threads places them.
template <int KT, int NT>
__device__ __forceinline__ void find_share(const PagedArgs &a, int min_pairs, Share *out) {
    __shared__ int64_t warp_sum[NT / 32];
    const int nb = a.prefix_phase ? 1 : a.B;
    const int run = (nb + NT - 1) / NT;
    const int b0 = min(nb, (int)threadIdx.x * run), b1 = min(nb, b0 + run);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = load_seq(a, b);
        mine += a.Hkv * key_tiles_before<KT>(a, s, row_tiles(a, s));
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if ((threadIdx.x & 31) >= o) incl += v;
    }
    if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < (int)(threadIdx.x >> 5)) before += warp_sum[w];
        total += warp_sum[w];
    }
    before += incl - mine;  // pairs of the runs before this thread's
    const int64_t fit = (total + min_pairs - 1) / min_pairs;
    const int ctas = fit < (int64_t)gridDim.x ? (int)fit : (int)gridDim.x;
    const bool some = (int)blockIdx.x < ctas;
    const int64_t begin = some ? share_begin(total, ctas, blockIdx.x) : total;
    if (some && begin >= before && begin < before + mine) {
        int64_t at = before;
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const Seq s = load_seq(a, b);
            const int64_t n = a.Hkv * key_tiles_before<KT>(a, s, row_tiles(a, s));
            if (begin < at + n) break;
            at += n;
        }
        out->seq = b;
        out->seq_begin = at;
    }
    if (threadIdx.x == 0) {
        out->total = total;
        out->ctas = ctas;
        out->begin = begin;
        out->end = some ? share_begin(total, ctas, blockIdx.x + 1) : total;
    }
    __syncthreads();
}

// The keys that token `tok` (piece token index i) attends to end before this.
__device__ __forceinline__ int row_limit(const PagedArgs &a, const Piece &p, int i) {
    if (!a.prefix_phase) return p.pos0 + i + 1;
    const int tok = p.tok0 + i;
    int lo = 0, hi = a.B - 1;  // the last sequence that starts at or before tok ...
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (__ldg(a.q_start + mid) <= tok) lo = mid;
        else hi = mid - 1;
    }
    // (empty sequences start where the next one does: the last of them is it)
    const int kv = min(max(__ldg(a.kv_len + lo), 0), a.cap);
    const int end = min(max(__ldg(a.q_start + lo + 1), 0), a.T);
    return min(a.prefix_len, kv - end + tok + 1);
}

// N consecutive output columns of one row, from its maximum m (log2 units),
// sum l and unnormalised output o: the prefix's buffer, or the output joined
// with it.  row = token * Hq + query head.
template <int D, int N>
__device__ __forceinline__ void write_row(const PagedArgs &a, int64_t row, int col, float m,
                                          float l, float (&o)[N]) {
    if (a.prefix_phase) {
        if (col == 0) a.prefix_ml[row] = make_float2(m, l);
        float4 *d = reinterpret_cast<float4 *>(a.prefix_o + row * D + col);
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            d[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        return;
    }
    float own = 1.0f;
    if (a.prefix_len > 0) {
        const float2 f = a.prefix_ml[row];
        const float top = fmaxf(m, f.x);
        own = max_factor(m, top);
        const float front = max_factor(f.x, top);
        l = l * own + f.y * front;
        const float4 *d = reinterpret_cast<const float4 *>(a.prefix_o + row * D + col);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = d[i];
            o[4 * i] = o[4 * i] * own + v.x * front;
            o[4 * i + 1] = o[4 * i + 1] * own + v.y * front;
            o[4 * i + 2] = o[4 * i + 2] * own + v.z * front;
            o[4 * i + 3] = o[4 * i + 3] * own + v.w * front;
        }
    }
    const float inv = l > 0.0f ? __frcp_rn(l) : 0.0f;  // no key: zeros
    float4 *d = reinterpret_cast<float4 *>(a.O + row * D + col);
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        d[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv,
                           o[4 * i + 3] * inv);
}

}  // namespace

// Launchers of the two kernels (see the files): the map of K and of V, one box
// of `bx` cache rows x 64 elements.
sq_status launch_paged_rows(const PagedArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                            int D, bool bf16, int row_groups, int bx, int sms, cudaStream_t st);

}  // namespace sq
