// Attention over the paged int8 cache for few query rows per key/value head: the
// single tokens and short drafts of a decoding step.
//
// A cached key row is k_scale codes, a value row v_scale codes, so with y = Q . codes
//   logit = y k_scale,  p = 2^(logit - m),  l += p,  O += (p v_scale) codes:
// the scales stand at the logits and the probabilities, the codes enter the products
// as they are.  The rest is paged_rows.cu's: a worker is a warp with a ring of its own,
// filled with cp.async by steps of 32 keys, products on the warp-level tensor
// instructions (m16n8k16), the running maximum, the pieces' join.
//
// Half the cache's bytes per key leave half the time for each, so the codes' way into
// the instruction's operands is kept short.  Which element of the contraction stands
// where in an operand is free, as long as both operands agree:
//   keys: thread t of a row's four takes the 16 bytes of chunk t (and t + 4) with one
//     load, four elements of them per instruction; the queries lie to match;
//   values: column n of an instruction's result is element D/8 n + i in its i-th
//     instruction, so that a thread's columns of all of them are 16 (8) bytes in a row.
// Codes become fp16 numbers exactly: a byte code + 128 in the low half of 0x6400 is
// 1024 + code + 128, from which 1152 is taken away, two codes at a time.
//
// Bound: memory and instruction issue together.  64 single tokens of 32 / 8 heads of 128,
// contexts to 8192: 104 us, 5.2 TB/s (78 % of the measured copy rate) at 46 % of the issue
// slots; steps of 16 keys 124 us, sums one by one instead of in pairs 106.  4 tokens of 64
// sequences of 4000 keys (16 rows): 176 us (200), the widening and twice the products.
//
// Precision: codes are exact in fp16; fp32 queries and weights p v_scale are sums of two
// fp16 numbers, each row scaled by a power of two so that its largest is within
// [2^7, 2^15) (queries) and [2^14, 2^15) (a step's weights), and what is 2^-37 of the
// row's largest weight still counts (see drop_zero_rows).  Logits are multiplied by a power
// of two as in paged_rows.cu.
#include "paged_rows.cuh"

#include <algorithm>
#include <mutex>

namespace sq {
namespace {

constexpr int kKT = kRowsI8Step;  // keys per step
constexpr int kWarps = 8;
constexpr int kPad = 1;       // an item's start and end, in steps
constexpr int kMinSteps = 2;  // steps of a worker's share at least
constexpr int kJoin = 16;     // pieces of an item that are joined in one go
constexpr int kPieces = 8;    // more than the steps that the copies are ahead

template <int D>
struct RowsI8Cfg {
    static constexpr int kCodes = kKT * D;                       // bytes of the keys or values
    static constexpr int kStepBytes = 2 * kCodes + 2 * kKT * 4;  // and both scales
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kSmem = kWarps * kStages * kStepBytes;
    static_assert(kStages < kPieces, "a piece per step in flight and the one being worked on");
};

// Byte offset of 16-byte chunk `ch` of row r: the reads below (four chunks of two
// neighbouring rows; two chunks of four rows of one parity) meet every bank once.
template <int D>
__device__ __forceinline__ int place(int r, int ch) {
    if (D == 128) return r * 128 + ((ch ^ ((r >> 1 & 3) << 1) ^ ((r & 1) << 2)) << 4);
    const int line = r >> 1;
    return line * 128 + ((((r & 1) << 2 | ch) ^ ((line & 3) << 1)) << 4);
}

__device__ __forceinline__ float lds_f1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// A value row of zeros adds nothing whatever its scale is (the append stores 1), but its
// weight could be the largest of a step, next to which the others' lose their parts.  So
// rows with scales above `known` are looked at: the scale of one of zeros becomes 0 (unless
// it is not finite: its products are NaN), and 2^8 times the largest of the others that
// are `seen` is known from then on.  Lane l: key l of the step.
template <int D>
__device__ __noinline__ float drop_zero_rows(uint32_t values, uint32_t scales, bool seen,
                                             float known) {
    static_assert(kKT == 32, "a key per lane");
    const int lane = threadIdx.x & 31;
    const float x = fabsf(lds_f1(scales + 4 * lane));
    const bool look = x > known && x < INFINITY;
    bool zeros = look;
#pragma unroll 1
    for (int ch = 0; ch < D / 16 && __any_sync(0xffffffffu, zeros); ++ch) {
        uint32_t w[4];
        lds4(w, values + place<D>(lane, ch));
        zeros = zeros && (w[0] | w[1] | w[2] | w[3]) == 0;
    }
    if (zeros)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + 4 * lane), "f"(0.0f) : "memory");
    __syncwarp();
    const float y = look && !zeros && seen ? 0x1p8f * x : 0.0f;
    return fmaxf(known, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(y))));
}
__device__ __forceinline__ float2 lds_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 1)
    paged_rows_i8_kernel(const __grid_constant__ PagedArgs a, const int8_t *__restrict__ k_cache,
                         const int8_t *__restrict__ v_cache) {
    using C = RowsI8Cfg<D>;
    using F = Parts<false, ROWS>;
    constexpr int ST = C::kStages, R = F::kRows, S = F::kSets;
    constexpr int NT = D / 8;  // a thread's columns of each of its two column groups
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
    int head_row = 0;  // the piece's head, in cache rows of a page
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
                head_row = p.head << a.page_shift;
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
            // the step's two blocks of 16 rows: each lies in a page, contiguous in the cache
            const int in_page = kr.key & ((1 << a.page_shift) - 1);
            const int second = (kr.key + 16) >> a.page_shift;
            constexpr int kLanes = D / 16, kCopies = C::kCodes / 1024, kStride = 32 / kLanes;
            const int r0 = lane / kLanes, ch = lane % kLanes;
            const uint32_t dst = ring + buf * C::kStepBytes;
            holes &= ~(3u << 2 * buf);
            int rows[2];  // (a cache has 2^30 at most)
            bool there[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // (both entries are in the lanes: a step begins at an even one or in a page)
                const int e = __shfl_sync(0xffffffffu, entry, (h ? second : idx) & 31);
                there[h] = e >= 0 && e < a.num_pages;
                holes |= (there[h] ? 0u : 1u) << (2 * buf + h);
                const int at = h && second != idx ? 0 : in_page + 16 * h;
                rows[h] = there[h] ? ((e * a.Hkv) << a.page_shift) + head_row + at : 0;
                // lane: chunk lane % kLanes of row lane / kLanes of every kStride rows.  (Rows
                // of no key are masked whatever they hold: codes are finite.)
                const int64_t from = (int64_t)rows[h] * D + lane * 16;
                const int8_t *ks = k_cache + from, *vs = v_cache + from;
#pragma unroll
                for (int j = 0; j < kCopies; ++j) {
                    const uint32_t d = dst + place<D>(16 * h + r0 + j * kStride, ch);
                    copy16(d, ks + j * 512, there[h]);
                    copy16(d + C::kCodes, vs + j * 512, there[h]);
                }
            }
            if (lane < 2 * kKT / 4)
                copy16(dst + 2 * C::kCodes + lane * 16,
                       (lane < kKT / 4 ? a.k_scale : a.v_scale) +
                           (lane & 4 ? rows[1] : rows[0]) + lane % 4 * 4,
                       lane & 4 ? there[1] : there[0]);
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
                      (p.head * a.G + row % a.G) * D + 16 * t;
        }
        auto out_row = [&](int r) {
            return (int64_t)(p.tok0 + tok[r]) * a.Hq + p.head * a.G + (g + 8 * r) % a.G;
        };
        // elements 64 c + 16 t + 4 i .. + 3 of row r's query
        auto query = [&](int r, int c, int i) {
            return live[r] ? *reinterpret_cast<const float4 *>(qrow[r] + 64 * c + 4 * i)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        float mul[R], scale[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float4 q = query(r, i / 4, i % 4);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)), fmaxf(fabsf(q.z), fabsf(q.w))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top *= fabsf(a.q_factor);
            const int sh = shift_of_wide((int)(__float_as_uint(top) >> 23) - 127, a.scale);
            mul[r] = a.q_factor * pow2(-sh);
            scale[r] = a.scale * pow2(sh);
        }
        uint32_t qf[D / 16][S][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            float x[2][R][2];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q = query(r, i / 4, i % 4);
                x[0][r][0] = q.x * mul[r];
                x[0][r][1] = q.y * mul[r];
                x[1][r][0] = q.z * mul[r];
                x[1][r][1] = q.w * mul[r];
            }
            F::fill(x[0], 0, qf[i]);
            F::fill(x[1], 2, qf[i]);
        }
        // o[i][r]: row r's elements NT 2 t + i and NT (2 t + 1) + i
        unsigned long long o[NT][R];
        float m[R], l[R];
        // four columns of row r from its element i of group q, and back
        auto four = [&](int r, int q, int i) {
            float x[4], y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) upk(o[i + k][r], x[k], y[k]);
            return q ? make_float4(y[0], y[1], y[2], y[3]) : make_float4(x[0], x[1], x[2], x[3]);
        };
        auto set_four = [&](int r, int q, int i, float4 v) {
            const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float x, y;
                upk(o[i + k][r], x, y);
                o[i + k][r] = q ? pk(x, w[k]) : pk(w[k], y);
            }
        };
        auto each_column = [&](auto &&f) {  // f(i of four columns, q, their first)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < NT; i += 4) f(i, q, NT * (2 * t + q) + i);
        };
#pragma unroll
        for (int i = 0; i < NT * R; ++i) o[i / R][i % R] = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
            if (live[r] && starts_with_prefix(a, p)) {
                const int64_t row = out_row(r);
                const float2 f = __ldcg(a.prefix_ml + row);
                m[r] = f.x;
                l[r] = t == 0 ? f.y : 0.0f;  // (the row's four threads' sums are added)
                each_column([&](int i, int q, int d) {
                    set_four(r, q, i,
                             __ldcg(reinterpret_cast<const float4 *>(a.prefix_o + row * D + d)));
                });
            }
        }
        int key0 = p.key0;
        float known = 0.0f;  // see drop_zero_rows
        for (int it = 0; it < p.ntiles; ++it, key0 += kKT) {
            asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
            __syncwarp();
            const uint32_t ks = ring + cur * C::kStepBytes;
            const uint32_t vs = ks + C::kCodes, sc = ks + 2 * C::kCodes;
            // (us with it here, behind the mask, and without: decode above 104, 104 and 103,
            // heads of 64 132, 129 and 126, 16 rows 176, 179 and 167)
            auto check_scales = [&]() {
                if (__any_sync(0xffffffffu, fabsf(lds_f1(sc + (kKT + lane) * 4)) > known)) {
                    const KeyRange kr = key_range(a, key0, p.keys);
                    const int k = kr.key + lane;
                    known = drop_zero_rows<D>(vs, sc + kKT * 4, kr.lo <= k && k < kr.hi, known);
                }
            };
            if (R > 1) check_scales();
            // logits of the rows x 32 keys
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i >> 2][i & 3] = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t w[4][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) lds4(w[h], ks + place<D>(g + 8 * h, t + 4 * c));
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t b = w[h][i] ^ kCodeBias;
                        const uint32_t b0 = fp16_codes(b, kCodesLow), b1 = fp16_codes(b, kCodesHigh);
#pragma unroll
                        for (int j = 0; j < S; ++j)
                            mma16816<false>(s[h], qf[4 * c + i][j], b0, b1);
                    }
            }
            // x[row][key]: element 2 h + b is key 8 h + 2 t + b of the step
            float x[R][8], vf[8];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float2 k2 = lds_f2(sc + (8 * h + 2 * t) * 4);
                if (R == 1) {
                    x[0][2 * h] = (s[h][0] + s[h][2]) * k2.x;
                    x[0][2 * h + 1] = (s[h][1] + s[h][3]) * k2.y;
                } else {
                    x[0][2 * h] = s[h][0] * k2.x;
                    x[0][2 * h + 1] = s[h][1] * k2.y;
                    x[R - 1][2 * h] = s[h][2] * k2.x;
                    x[R - 1][2 * h + 1] = s[h][3] * k2.y;
                }
            }
            // keys that are masked: behind the row's own, in front of the
            // suffix, or of a page that is missing
            const KeyRange kr = key_range(a, key0, limit[0]);
            const int hi1 = R == 1 ? 0 : key_range(a, key0, limit[R - 1]).hi;
            const unsigned missing = holes >> 2 * cur & 3u;
            bool cut = kr.key < kr.lo || kr.key + kKT > kr.hi ||
                       (R > 1 && kr.key + kKT > hi1) || missing;
            cut = __any_sync(0xffffffffu, cut);
            if (cut) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = kr.key + 8 * (i >> 1) + 2 * t + (i & 1);
                        if ((missing >> (i >> 2) & 1) || k >= (r ? hi1 : kr.hi) || k < kr.lo)
                            x[r][i] = -INFINITY;
                    }
            }
            if (R == 1) check_scales();
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float2 v2 = lds_f2(sc + (kKT + 8 * h + 2 * t) * 4);
                vf[2 * h] = v2.x;
                vf[2 * h + 1] = v2.y;
            }
            float grow[R];
            bool any = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mx = x[r][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[r][i]);
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
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) o[i][r] = mul2(o[i][r], pk(grow[r], grow[r]));
            }
            uint32_t pf[2][S][4];  // of the step's two blocks of 16 keys
            unsigned long long down2[R];
            {
                float w[4][R][2];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float from = m[r] == -INFINITY ? 0.0f : -m[r];  // (no key yet)
                    float top = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float pr = ex2(fmaf(x[r][i], scale[r], from));
                        l[r] += pr;
                        // (a masked key's scale need not be finite)
                        w[i >> 1][r][i & 1] = cut && x[r][i] == -INFINITY ? 0.0f : pr * vf[i];
                        top = fmaxf(top, fabsf(w[i >> 1][r][i & 1]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // the row's largest weight into [2^14, 2^15)
                    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100) - 14;
                    const float up = pow2(-e);
                    down2[r] = pk(pow2(e), pow2(e));
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i >> 1][r][i & 1] *= up;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    F::fill(w[2 * h], 0, pf[h]);
                    F::fill(w[2 * h + 1], 2, pf[h]);
                }
            }
            // the values of this thread's keys, NT bytes of each: v[h][i] of key 8 (2 h + i / 2)
            // + 2 t + i % 2
            constexpr int NW = NT / 4;
            uint32_t v[2][4][NW];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 8 * (i >> 1) + 2 * t + (i & 1);
                uint32_t (&y)[NW] = v[i >> 2][i & 3];
                if constexpr (D == 128) {
                    lds4(y, vs + place<D>(r, g));
                } else {
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                                 : "=r"(y[0]), "=r"(y[1])
                                 : "r"(vs + place<D>(r, g >> 1) + 8 * (g & 1))
                                 : "memory");
                }
#pragma unroll
                for (int j = 0; j < NW; ++j) y[j] ^= kCodeBias;
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                // byte i of keys 2 t and 2 t + 1, and of 2 t + 8 and 2 t + 9
                const int j = i / 4;
                const uint32_t pair = i & 2 ? 0x7362u : 0x5140u;
                const uint32_t half = i & 1 ? kCodesHigh : kCodesLow;
                // (the instruction's accumulator truncates: the step's products alone go
                // through it)
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t b0 = fp16_codes(__byte_perm(v[h][0][j], v[h][1][j], pair), half);
                    const uint32_t b1 = fp16_codes(__byte_perm(v[h][2][j], v[h][3][j], pair), half);
#pragma unroll
                    for (int k = 0; k < S; ++k) mma16816<false>(c, pf[h][k], b0, b1);
                }
                if (R == 1) {
                    o[i][0] = fma2(add2(pk(c[0], c[1]), pk(c[2], c[3])), down2[0], o[i][0]);
                } else {
                    o[i][0] = fma2(pk(c[0], c[1]), down2[0], o[i][0]);
                    o[i][R - 1] = fma2(pk(c[2], c[3]), down2[R - 1], o[i][R - 1]);
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
                    each_column([&](int i, int q, int d) {
                        __stcg(reinterpret_cast<float4 *>(a.part_o + (at + 8 * r) * D + d),
                               four(r, q, i));
                    });
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
                    for (int i = 0; i < NT; ++i) o[i][r] = 0;
#pragma unroll 2
                    for (int c = 0; c < join.n; ++c) {
                        const int64_t base = part_row(join.first + c * join.step) + 8 * r;
                        const float2 f = __ldcg(a.part_ml + base);
                        const float top = fmaxf(m[r], f.x);
                        const float fo = max_factor(m[r], top), fp = max_factor(f.x, top);
                        m[r] = top;
                        l[r] = l[r] * fo + f.y * fp;
                        each_column([&](int i, int q, int d) {
                            const float4 v =
                                __ldcg(reinterpret_cast<const float4 *>(a.part_o + base * D + d));
                            const float4 w = four(r, q, i);
                            set_four(r, q, i,
                                     make_float4(w.x * fo + v.x * fp, w.y * fo + v.y * fp,
                                                 w.z * fo + v.z * fp, w.w * fo + v.w * fp));
                        });
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
            float *dst = row_target(a) + row * D;
            each_column([&](int i, int q, int d) {
                const float4 v = four(r, q, i);
                *reinterpret_cast<float4 *>(dst + d) =
                    make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            });
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int ROWS>
sq_status launch_rows_i8(const PagedArgs &a, const void *k_cache, const void *v_cache, int sms,
                         cudaStream_t st) {
    using C = RowsI8Cfg<D>;
    static std::mutex mu;
    static bool done[64] = {};
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[di.device & 63]) {
            if (cudaFuncSetAttribute(paged_rows_i8_kernel<D, ROWS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::kSmem) != cudaSuccess)
                return SQ_ERR_CUDA;
            done[di.device & 63] = true;
        }
    }
    return launch_pdl(paged_rows_i8_kernel<D, ROWS>, dim3((unsigned)sms), dim3(kWarps * 32),
                      C::kSmem, st, 1, a, static_cast<const int8_t *>(k_cache),
                      static_cast<const int8_t *>(v_cache));
}

}  // namespace

sq_status launch_paged_rows_i8(const PagedArgs &a, const void *k_cache, const void *v_cache, int D,
                               int rows, int sms, cudaStream_t st) {
    if (D == 128)
        return rows == 8 ? launch_rows_i8<128, 8>(a, k_cache, v_cache, sms, st)
                         : launch_rows_i8<128, 16>(a, k_cache, v_cache, sms, st);
    return rows == 8 ? launch_rows_i8<64, 8>(a, k_cache, v_cache, sms, st)
                     : launch_rows_i8<64, 16>(a, k_cache, v_cache, sms, st);
}

}  // namespace sq
