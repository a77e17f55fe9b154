// Shared parts of the attention kernels over the paged cache: the workers'
// shares, the split of fp32 numbers over 16-bit ones, and the rows' last step.
#pragma once
#include "decoder.cuh"
#include "paged_line.cuh"

#include <cuda_fp16.h>

namespace sq {

namespace {

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

// 2^e, e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// The multiple of 8 that scales numbers whose largest has the exponent e into
// fp16's range, the largest into [2^7, 2^15) (fp16 ends at 65504, so the octave
// below 2^16 would round to infinity at its end); tiny and zero rows as if e = -32.
__device__ __forceinline__ int shift_of(int e) { return (max(e, -32) - 7) & ~7; }

// N pairs of 16-bit numbers of the cache's type that sum to (a, b), a in the
// low half.  Three bf16 numbers hold an fp32 number exactly: each takes the
// next 8 bits of its significand, by masking (the conversion instructions run
// at a quarter of the rate).  Two fp16 numbers are within 2^-22 of it, each the
// rounding of what is left.
template <bool BF, int N>
__device__ __forceinline__ void split16(float a, float b, uint32_t (&w)[N]) {
    static_assert(N == (BF ? 3 : 2), "parts of an fp32 number");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (BF) {
            const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
            w[i] = __byte_perm(ua, ub, 0x7632);  // the two high halves
            if (i + 1 < N) {
                a -= __uint_as_float(ua & 0xffff0000u);
                b -= __uint_as_float(ub & 0xffff0000u);
            }
        } else {
            const __half2 h = __floats2half2_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
            a -= __low2float(h);
            b -= __high2float(h);
        }
    }
}

// 16 bytes of global memory into shared memory, asynchronously, or zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void lds4(uint32_t (&w)[4], uint32_t addr) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}
// Bits 15 and 31: the 16-bit numbers of the pair that are not finite (an exponent
// of ones; adding its lowest bit carries into the sign's place).
template <bool BF>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return ((w & (BF ? 0x7f807f80u : 0x7c007c00u)) + (BF ? 0x00800080u : 0x04000400u)) &
           0x80008000u;
}
// the pair with zeros in their places
template <bool BF>
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
    const uint32_t f = not_finite<BF>(w);
    return w & ((f & 0x8000u ? 0u : 0xffffu) | (f >> 31 ? 0u : 0xffff0000u));
}
template <bool BF>
__device__ __forceinline__ float widen16(uint32_t low) {
    return BF ? __uint_as_float(low << 16) : __half2float(__ushort_as_half((uint16_t)low));
}

// The line's length and the shares of this block's W workers (worker w of block
// c is number w gridDim.x + c, so that neighbours on the line are on different
// SMs), by all NT threads: each sums a run of sequences, a scan over the
// threads places them.
template <int KT, int PAD, int NT, int W>
__device__ __forceinline__ void find_shares(const PagedArgs &a, int min_pairs, Share *out) {
    __shared__ int warp_sum[NT / 32];
    const int nb = a.prefix_phase ? 1 : a.B;
    const int run = (nb + NT - 1) / NT;
    const int b0 = min(nb, (int)threadIdx.x * run);
    int b1 = min(nb, b0 + run);
    int mine = 0, before = 0;
    bool overlap = false;  // (the sums may wrap around then, and are not used)
    // first every thread's run is summed, then the shares that begin in it are
    // found, walking through it again
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        int at = before;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const Seq s = load_seq(a, b);
            const int n = a.Hkv * pairs_before<KT, PAD>(a, s, row_tiles(a, s));
            if (pass == 0) {
                mine += n;
                overlap = overlap || !in_order(a, b);
                continue;
            }
#pragma unroll 1
            for (int w = 0; w < W; ++w)
                if (out[w].begin >= at && out[w].begin < at + n) {
                    out[w].seq = b;
                    out[w].seq_begin = at;
                }
            at += n;
        }
        if (pass == 1) break;
        int incl = mine;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if ((threadIdx.x & 31) >= o) incl += v;
        }
        if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = incl;
        const bool none = __syncthreads_or(overlap) != 0;
        int total = 0;
#pragma unroll 1
        for (int w = 0; w < NT / 32; ++w) {
            if (w < (int)(threadIdx.x >> 5)) before += warp_sum[w];
            total += warp_sum[w];
        }
        if (none) {
            total = 0;
            b1 = b0;  // no share has a place
        }
        before += incl - mine;  // pairs of the runs before this thread's
        if (threadIdx.x < W) {
            int workers = min((total + min_pairs - 1) / min_pairs, W * (int)gridDim.x);
            if (a.prefix_phase && total > 0) {
                // items of one length: whole numbers of workers for each, where
                // there are enough, so that no worker has parts of two
                const int items = total / key_tiles<KT>(a, load_seq(a, 0), 0);
                if (items < workers) workers -= workers % items;
            }
            set_shares(out[threadIdx.x], total, workers,
                       (int)threadIdx.x * (int)gridDim.x + (int)blockIdx.x);
        }
        __syncthreads();
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

// Where a row of an item starts: with no key, or, at the suffix's first key, with
// the prefix's maximum, sum and output (so that its loads are on their way while
// the item's first keys are).  row = token * Hq + query head.
__device__ __forceinline__ bool starts_with_prefix(const PagedArgs &a, const Piece &p) {
    return !a.prefix_phase && a.prefix_len > 0 && a.front_tiles == 0 && p.key0 == a.kstart;
}
// A row's last step, from its maximum m (log2 units) and sum l: the factor of its
// output on the way to the prefix's buffer (with m and l, stored by the caller
// that is `first`) or to the result.
__device__ __forceinline__ float row_factor(const PagedArgs &a, int64_t row, float m, float l,
                                            bool first) {
    if (a.prefix_phase) {
        if (first) a.prefix_ml[row] = make_float2(m, l);
        return 1.0f;
    }
    return l > 0.0f ? __frcp_rn(l) : 0.0f;  // no key: zeros
}
__device__ __forceinline__ float *row_target(const PagedArgs &a) {
    return a.prefix_phase ? a.prefix_o : a.O;
}

}  // namespace

// The kernel for at most 16 rows per item (paged_rows.cu): rows = 8 or 16.
sq_status launch_paged_rows(const PagedArgs &a, const void *k_cache, const void *v_cache, int D,
                            bool bf16, int rows, int sms, cudaStream_t st);
// The kernel for up to 128 rows per item (paged_tiles.cu).
sq_status launch_paged_tiles(const PagedArgs &a, const void *k_cache, const void *v_cache, int D,
                             bool bf16, int sms, cudaStream_t st);

}  // namespace sq
