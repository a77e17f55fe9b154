// Attention over the paged cache for few query rows per key/value head: the
// single tokens and short drafts of a decoding step.
//
// With m the running row maximum and l the running sum (both fp32), a tile of
// keys contributes s = q K^T, m' = max(m, max s), p = 2^(s - m'), and
// l = l 2^(m - m') + sum p, O = O 2^(m - m') + p V: one pass over the cache.
// Every byte of the cache serves at most 16 rows, so the kernel is bound by
// memory; all it has to do is keep enough copies in flight and the arithmetic
// out of their way.
//
// A worker is a warp: it takes its share of the line in steps of 16 keys, with
// a ring of its own in shared memory that it fills with cp.async, two or more
// steps ahead and across the borders of items.  Warps meet nobody, so that no
// warp's item end stalls the others' copies; 8 warps hold 128 KB in flight per
// SM.  A step lies in one page whatever the page's size (TMA boxes of one
// 16-row page each measured 104 ns of its unit's time a box, 3.0 TB/s in all;
// 16-byte copies by the lanes stream random 16-row pages at 7.0 TB/s).  Rows
// behind the last key and rows of missing pages are filled with zeros.
//
// The products run on the warp-level tensor instructions (m16n8k16, 8 cycles
// each per SM quarter): 16 rows are too few for tensor memory's 128.
//
// Measured (32 / 8 heads of 128, bf16): a step of 64 sequences of up to 8192 keys
// 161 us, 6.5 TB/s, 96 % of the measured copy rate; one token behind 300 keys 14
// us, behind 4000 21, behind 100,000 83 (4.8 TB/s): those are bound by latency, the
// start's chain of dependent loads and the pieces' join.
//
// Precision: keys and values enter as stored.  The fp32 queries and
// probabilities are split over several 16-bit numbers (split16): two for fp16
// (within 2^-22, or 2^-32 of a row's largest), three for bf16 (exact).  Fp16's
// probabilities carry a factor 2^12: its smallest step is 2^-24, and without it a
// key of less than 2^-25 of the largest's weight would count in the sum alone (8192
// of 2^-25 behind one of 1: 2.3e-4 of the output, all of what they say).  The queries
// carry the scale's significand, so that logits are multiplied by a power of two:
// the largest key's exponent is 0 however large its logit is.
// Up to 8 rows, two of the parts share an instruction's 16 rows (the first in
// rows 0-7, the second in rows 8-15) and the two halves are added in fp32.
#include "paged.cuh"

#include <algorithm>
#include <mutex>

namespace sq {
namespace {

constexpr int kKT = 16;       // keys per step
constexpr int kWarps = 8;
constexpr int kPad = 2;       // an item's start and end, in steps
// Steps of a worker's share at least: 4, 6 and 10 measured 15, 17 and 19 us (one
// token, 300 or 600 keys)
constexpr int kMinSteps = 4;
// Pieces of an item that are joined in one go (0.2 us each): 8, 16 and 32 measured
// 27, 27 and 31 us (8 tokens, 2000 keys); all in one go took 298 instead of 40 us
// for one key/value head's 100,000 keys
constexpr int kJoin = 16;
constexpr int kPieces = 8;    // more than the steps that the copies are ahead

constexpr float kUp = 4096.0f;  // fp16 probabilities' factor

template <int D>
struct RowsCfg {
    static constexpr int kStepBytes = 2 * kKT * D * 2;  // keys, then values
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kSmem = kWarps * kStages * kStepBytes;
    static_assert(kStages < kPieces, "a piece per step in flight and the one being worked on");
};

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The instruction's operand sets for rows of which each thread holds RPT (ROWS
// / 8) pairs of elements: N parts of ROWS = 8 rows in (N + 1) / 2 sets, of 16
// rows in N sets.
template <bool BF, int ROWS>
struct Parts {
    static constexpr int kParts = BF ? 3 : 2;
    static constexpr int kSets = ROWS == 8 ? (kParts + 1) / 2 : kParts;
    static constexpr int kRows = ROWS / 8;
    // registers r and r + 1 of every set (rows 0-7 and 8-15) from this thread's
    // pairs (x[row][0], x[row][1])
    static __device__ __forceinline__ void fill(const float (&x)[kRows][2], int r,
                                                uint32_t (&f)[kSets][4]) {
        uint32_t w[kRows][kParts];
#pragma unroll
        for (int i = 0; i < kRows; ++i) split16<BF, kParts>(x[i][0], x[i][1], w[i]);
        if (ROWS == 8) {
            f[0][r] = w[0][0];
            f[0][r + 1] = w[0][1];
            if (kSets > 1) {
                f[kSets - 1][r] = w[0][kParts - 1];
                f[kSets - 1][r + 1] = 0;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSets; ++j) {
                f[j][r] = w[0][j];
                f[j][r + 1] = w[kRows - 1][j];
            }
        }
    }
};

// The order of launches.  The prefix's launch, of either kernel, lets the next one
// start only when the kernels before it are complete, so that the launch behind it
// (after_prefix) need not wait for them, but for the prefix's state and the workspace
// alone (end_of_prefix, in front of the first access to either); its first copies
// are on their way meanwhile: 4 us less of 70 to 140.  (The kernel for many rows
// gains nothing: 117 us either way.)
__device__ __forceinline__ void begin_rows(const PagedArgs &a) {
    if (!a.prefix_phase) pdl_launch_dependents();
    if (!a.after_prefix) pdl_wait();  // the accesses below follow the previous kernel
    if (a.prefix_phase) pdl_launch_dependents();
}
__device__ __forceinline__ void end_of_prefix(const PagedArgs &a) {
    if (a.after_prefix) pdl_wait();
}

template <int D, bool BF, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 1)
    paged_rows_kernel(const __grid_constant__ PagedArgs a, const uint16_t *__restrict__ k_cache,
                      const uint16_t *__restrict__ v_cache) {
    using C = RowsCfg<D>;
    using F = Parts<BF, ROWS>;
    constexpr int ST = C::kStages, R = F::kRows, S = F::kSets;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Share shares[kWarps];
    __shared__ Piece pieces[kWarps][kPieces];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    begin_rows(a);
    find_shares<kKT, kPad, kWarps * 32, kWarps>(a, kMinSteps, shares);
    const Share &share = shares[warp];
    const int worker = warp * gridDim.x + blockIdx.x;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * ST * C::kStepBytes;

    // ---- the copies: one step of the share per call, or nothing at its end
    Walk<kKT, kPad> walk;
    walk.start(a, share);
    int npieces = 0, left = 0, key = 0, held = -1, entry = -1;
    int buf = 0;  // the ring's buffer that is filled next
    int64_t head_row = 0;  // the piece's head, in cache rows of a page
    int keys = 0;
    unsigned holes = 0;    // bit i: the page of the step in buffer i is missing
    const int *table = nullptr;
    auto copy_step = [&]() {
        if (left == 0) {
            Piece p;
            if (walk.next(a, share, p)) {
                if (lane == 0) pieces[warp][npieces % kPieces] = p;
                ++npieces;
                left = p.ntiles;
                key = p.key0;
                keys = p.keys;
                head_row = (int64_t)p.head << a.page_shift;
                table = a.block_table + (int64_t)p.seq * a.max_pages;
                held = -1;
            }
        }
        if (left > 0) {
            // lane i holds the page-table entry 32 held + i
            const KeyRange kr = key_range(a, key, keys);
            const int idx = kr.key >> a.page_shift;
            if (idx >> 5 != held || key == a.kstart) {
                held = idx >> 5;
                const int at = (held << 5) + lane;
                entry = (int64_t)at << a.page_shift < kr.hi
                            ? __ldg((kr.front ? a.prefix_pages : table) + at)
                            : -1;
            }
            const int e = __shfl_sync(0xffffffffu, entry, idx & 31);
            const bool there = e >= 0 && e < a.num_pages;
            holes = (holes & ~(1u << buf)) | (there ? 0u : 1u << buf);
            const int64_t row0 = (there ? (((int64_t)e * a.Hkv) << a.page_shift) + head_row : 0) +
                                 (kr.key & ((1 << a.page_shift) - 1));
            // lane: chunk lane % (D / 8) of row lane / (D / 8) of every kStride rows; the
            // step's 16 rows are contiguous in the cache
            constexpr int kLanes = D / 8, kCopies = kKT * kLanes / 32, kStride = 32 / kLanes;
            const int r0 = lane / kLanes, ch = lane % kLanes;
            const uint32_t dst = ring + buf * C::kStepBytes + r0 * D * 2;
            const int64_t from = row0 * D + lane * 8;
            const uint16_t *ks = k_cache + from, *vs = v_cache + from;
            if (there && kr.key + kKT <= kr.hi && kr.key >= kr.lo) {
#pragma unroll
                for (int j = 0; j < kCopies; ++j) {
                    const uint32_t d =
                        dst + j * 512 + (((ch ^ r0) ^ (j * kStride & 7)) << 4);
                    copy16(d, ks + j * 256, true);
                    copy16(d + kKT * D * 2, vs + j * 256, true);
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < kCopies; ++j) {
                    const int r = r0 + j * kStride;
                    const bool in = there && kr.key + r < kr.hi && kr.key + r >= kr.lo;
                    const uint32_t d =
                        dst + j * 512 + (((ch ^ r0) ^ (j * kStride & 7)) << 4);
                    copy16(d, in ? ks + j * 256 : k_cache, in);
                    copy16(d + kKT * D * 2, in ? vs + j * 256 : v_cache, in);
                }
            }
            key += kKT;
            --left;
        }
        if (++buf == ST) buf = 0;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) copy_step();
    end_of_prefix(a);
    __syncwarp();

    const int g = lane >> 2, t = lane & 3;  // fragment row and column pair
    int cur = 0;  // the ring's buffer of the step
    for (int n = 0; n < npieces; ++n) {
        const Piece p = pieces[warp][n % kPieces];
        // this thread's rows of the item: g and, of 16, g + 8
        int tok[R], limit[R];
        bool live[R];
        const float *qrow[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = g + 8 * i;
            tok[i] = row / a.G;
            live[i] = tok[i] < p.ntok;
            limit[i] = live[i] ? row_limit(a, p, tok[i]) : p.keys;
            qrow[i] = a.Q + (int64_t)(p.tok0 + tok[i]) * a.ldq +
                      (p.head * a.G + row % a.G) * D + 2 * t;
        }
        auto out_row = [&](int r) {
            return (int64_t)(p.tok0 + tok[r]) * a.Hq + p.head * a.G + (g + 8 * r) % a.G;
        };
        // fp16 queries are scaled row by row by a power of two into fp16's range
        float mul[R], scale[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mul[r] = a.q_factor;
            scale[r] = a.scale;
            if (BF) continue;
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 q = live[r] ? *reinterpret_cast<const float2 *>(qrow[r] + 8 * i)
                                         : make_float2(0.f, 0.f);
                top = fmaxf(top, fmaxf(fabsf(q.x), fabsf(q.y)));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top *= fabsf(a.q_factor);
            const int sh = shift_of((int)(__float_as_uint(top) >> 23) - 127);
            mul[r] *= pow2(-sh);
            scale[r] *= pow2(sh);
        }
        uint32_t qf[D / 16][S][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 q =
                        live[r] ? *reinterpret_cast<const float2 *>(qrow[r] + 16 * i + 8 * h)
                                : make_float2(0.f, 0.f);
                    x[r][0] = q.x * mul[r];
                    x[r][1] = q.y * mul[r];
                }
                F::fill(x, 2 * h, qf[i]);
            }
        float o[D / 8][2 * R], m[R], l[R];
#pragma unroll
        for (int i = 0; i < D / 8 * 2 * R; ++i) o[i / (2 * R)][i % (2 * R)] = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
            if (live[r] && starts_with_prefix(a, p)) {
                const int64_t row = out_row(r);
                const float2 f = __ldcg(a.prefix_ml + row);
                m[r] = f.x;
                l[r] = t == 0 ? f.y : 0.0f;  // (the row's four threads' sums are added)
                const float *src = a.prefix_o + row * D + 2 * t;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + 8 * i));
                    o[i][2 * r] = v.x;
                    o[i][2 * r + 1] = v.y;
                }
            }
        }
        int key0 = p.key0;
        for (int it = 0; it < p.ntiles; ++it, key0 += kKT) {
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
            __syncwarp();
            const uint32_t ks = ring + cur * C::kStepBytes;
            const uint32_t vs = ks + kKT * D * 2;
            // logits of the rows x 16 keys
            float s[2][2][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i >> 3][i >> 2 & 1][i & 3] = 0.0f;
            {
                const int kr = (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t b[4];
                    ldsm4(b, ks + kr * D * 2 + (((2 * i + half) ^ (kr & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < S; ++j) {
                        mma16816<BF>(s[i & 1][0], qf[i][j], b[0], b[1]);
                        mma16816<BF>(s[i & 1][1], qf[i][j], b[2], b[3]);
                    }
                }
            }
            // x[row][key]: keys 2t, 2t + 1, 2t + 8, 2t + 9 of the step
            float x[R][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float c0 = s[0][e >> 1][e & 1] + s[1][e >> 1][e & 1];
                const float c1 = s[0][e >> 1][2 + (e & 1)] + s[1][e >> 1][2 + (e & 1)];
                if (R == 1) x[0][e] = c0 + c1;
                else x[0][e] = c0, x[R - 1][e] = c1;
            }
            // keys that are masked: behind the row's own, in front of the
            // suffix, or of a page that is missing
            const KeyRange kr = key_range(a, key0, limit[0]);
            const int hi1 = R == 1 ? 0 : key_range(a, key0, limit[R - 1]).hi;
            bool cut = kr.key < kr.lo || kr.key + kKT > kr.hi ||
                       (R > 1 && kr.key + kKT > hi1);
            const bool missing = holes >> cur & 1;
            cut = __any_sync(0xffffffffu, cut);
            if (cut || missing) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = kr.key + 8 * (i >> 1) + 2 * t + (i & 1);
                        if (missing || k >= (r ? hi1 : kr.hi) || k < kr.lo) x[r][i] = -INFINITY;
                    }
            }
            float grow[R];
            bool any = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mx = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = mx == -INFINITY ? m[r] : fmaxf(m[r], mx * scale[r]);
                any = any || mn > m[r];
                grow[r] = mn > m[r] ? max_factor(m[r], mn) : 1.0f;
                m[r] = mn;
            }
            if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                for (int r = 0; r < R; ++r) l[r] *= grow[r];
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        o[i][2 * r] *= grow[r];
                        o[i][2 * r + 1] *= grow[r];
                    }
            }
            if (cut) {
                // a masked key's probability is zero, but its value need not be
                // finite, and zero times that is NaN: such values are added to the
                // rows that see them and taken out of the step
                constexpr int kChunks = kKT * D / 8 / 32;  // 16-byte chunks per lane
                uint32_t bad = 0;
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    uint32_t w[4];
                    lds4(w, vs + (i * 32 + lane) * 16);
                    bad |= not_finite<BF>(w[0]) | not_finite<BF>(w[1]) | not_finite<BF>(w[2]) |
                           not_finite<BF>(w[3]);
                }
                if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
                    for (int k = 0; k < kKT; ++k) {
                        const int at = kr.key + k;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];"
                                         : "=r"(w)
                                         : "r"(vs + k * D * 2 + ((i ^ (k & 7)) << 4) + 4 * t)
                                         : "memory");
                            const uint32_t f = not_finite<BF>(w);
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                if (at < kr.lo || at >= (r ? hi1 : kr.hi)) continue;
                                if (f & 0x8000u) o[i][2 * r] += widen16<BF>(w & 0xffffu);
                                if (f >> 31) o[i][2 * r + 1] += widen16<BF>(w >> 16);
                            }
                        }
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int i = 0; i < kChunks; ++i) {
                        uint32_t w[4];
                        lds4(w, vs + (i * 32 + lane) * 16);
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = finite_part<BF>(w[j]);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         vs + (i * 32 + lane) * 16),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                    __syncwarp();
                }
            }
            uint32_t pf[S][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float from = m[r] == -INFINITY ? 0.0f : -m[r];  // (no key yet)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[r][i] = ex2(fmaf(x[r][i], scale[r], from));
                    l[r] += x[r][i];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float y[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    y[r][0] = BF ? x[r][2 * h] : x[r][2 * h] * kUp;
                    y[r][1] = BF ? x[r][2 * h + 1] : x[r][2 * h + 1] * kUp;
                }
                F::fill(y, 2 * h, pf);
            }
            {
                const int kr = ((lane >> 3) & 1) * 8 + (lane & 7), half = lane >> 4;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t b[4];
                    ldsm4t(b, vs + kr * D * 2 + (((2 * i + half) ^ (kr & 7)) << 4));
                    // the step's products alone go through the instruction's
                    // accumulator, which truncates: over 512 steps that would
                    // cost 6e-6 of the output
                    float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int j = 0; j < S; ++j) {
                        mma16816<BF>(c[0], pf[j], b[0], b[1]);
                        mma16816<BF>(c[1], pf[j], b[2], b[3]);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            constexpr float kDown = BF ? 1.0f : 1.0f / kUp;
                            float &o0 = o[2 * i + j][q], &o1 = o[2 * i + j][2 * R - 2 + q];
                            if (R == 1) {
                                o0 = fmaf(c[j][q] + c[j][2 + q], kDown, o0);
                            } else {
                                o0 = fmaf(c[j][q], kDown, o0);
                                o1 = fmaf(c[j][2 + q], kDown, o1);
                            }
                        }
                }
            }
            __syncwarp();  // the step's buffer is free
            copy_step();
            if (++cur == ST) cur = 0;
        }
        __syncwarp();  // the copies' next piece is in shared memory
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        if (p.npieces > 1) {
            // this worker's part of the item; whoever is last of a group, and then of
            // the groups, joins them all
            auto part_row = [&](int c) {  // piece c of the item
                return (int64_t)(2 * (p.first + c) + (c == 0)) * ROWS + g;
            };
            auto put_part = [&](int64_t at) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float *d = a.part_o + (at + 8 * r) * D + 2 * t;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        __stcg(reinterpret_cast<float2 *>(d + 8 * i),
                               make_float2(o[i][2 * r], o[i][2 * r + 1]));
                    if (t == 0) __stcg(a.part_ml + at + 8 * r, make_float2(m[r], l[r]));
                }
            };
            const int width = join_width(p.npieces, kJoin);
            Join join = join_of(p, worker - p.first, width);
            bool joined = true;
            int64_t at = part_row(worker - p.first);
            for (;;) {
                put_part(at);
                __threadfence();
                __syncwarp();
                unsigned last = 0;
                if (lane == 0) {
                    last = atomicAdd(a.counters + join.counter, 1u) == (unsigned)join.n - 1;
                    if (last) a.counters[join.counter] = 0;  // as the next launch wants it
                }
                if (!__shfl_sync(0xffffffffu, last, 0)) {
                    joined = false;
                    break;
                }
                __threadfence();
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    m[r] = -INFINITY;
                    l[r] = 0.0f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) o[i][2 * r] = o[i][2 * r + 1] = 0.0f;
#pragma unroll 2
                    for (int c = 0; c < join.n; ++c) {
                        const int64_t base = part_row(join.first + c * join.step) + 8 * r;
                        const float2 f = __ldcg(a.part_ml + base);
                        const float top = fmaxf(m[r], f.x);
                        const float fo = max_factor(m[r], top), fp = max_factor(f.x, top);
                        m[r] = top;
                        l[r] = l[r] * fo + f.y * fp;
                        const float *src = a.part_o + base * D + 2 * t;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            const float2 v = __ldcg(reinterpret_cast<const float2 *>(src + 8 * i));
                            o[i][2 * r] = o[i][2 * r] * fo + v.x * fp;
                            o[i][2 * r + 1] = o[i][2 * r + 1] * fo + v.y * fp;
                        }
                    }
                }
                if (join.all) break;
                // the group's sum in the place of its first piece
                __syncwarp();
                at = part_row(join.first);
                join = join_of_groups(p, width);
            }
            if (!joined) continue;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!live[r]) continue;
            const int64_t row = out_row(r);
            const float f = row_factor(a, row, m[r], l[r], t == 0);
            float *dst = row_target(a) + row * D + 2 * t;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(dst + 8 * i) =
                    make_float2(o[i][2 * r] * f, o[i][2 * r + 1] * f);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, bool BF, int ROWS>
sq_status launch_rows(const PagedArgs &a, const void *k_cache, const void *v_cache, int sms,
                      cudaStream_t st) {
    using C = RowsCfg<D>;
    static std::mutex mu;
    static bool done[64] = {};
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[di.device & 63]) {
            if (cudaFuncSetAttribute(paged_rows_kernel<D, BF, ROWS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::kSmem) != cudaSuccess)
                return SQ_ERR_CUDA;
            done[di.device & 63] = true;
        }
    }
    return launch_pdl(paged_rows_kernel<D, BF, ROWS>, dim3((unsigned)sms), dim3(kWarps * 32),
                      C::kSmem, st, 1, a, static_cast<const uint16_t *>(k_cache),
                      static_cast<const uint16_t *>(v_cache));
}

}  // namespace

sq_status launch_paged_rows(const PagedArgs &a, const void *k_cache, const void *v_cache, int D,
                            bool bf16, int rows, int sms, cudaStream_t st) {
    const int v = (D == 128 ? 4 : 0) + (bf16 ? 2 : 0) + (rows == 16 ? 1 : 0);
    switch (v) {
    case 0: return launch_rows<64, false, 8>(a, k_cache, v_cache, sms, st);
    case 1: return launch_rows<64, false, 16>(a, k_cache, v_cache, sms, st);
    case 2: return launch_rows<64, true, 8>(a, k_cache, v_cache, sms, st);
    case 3: return launch_rows<64, true, 16>(a, k_cache, v_cache, sms, st);
    case 4: return launch_rows<128, false, 8>(a, k_cache, v_cache, sms, st);
    case 5: return launch_rows<128, false, 16>(a, k_cache, v_cache, sms, st);
    case 6: return launch_rows<128, true, 8>(a, k_cache, v_cache, sms, st);
    default: return launch_rows<128, true, 16>(a, k_cache, v_cache, sms, st);
    }
}

}  // namespace sq
