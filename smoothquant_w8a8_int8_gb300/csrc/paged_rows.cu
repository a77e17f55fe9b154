// Attention over the paged cache for few query rows per key/value head: the
// single tokens and short drafts of a decoding step.
//
// With m the running row maximum and l the running sum (both fp32), a tile of
// keys contributes s = q K^T, m' = max(m, max s), p = 2^(s - m'), and
// l = l 2^(m - m') + sum p, O = O 2^(m - m') + p V: one pass over the cache.
// The cache is read once and every byte of it serves at most 16 rows, so the
// kernel is bound by memory; all it has to do is keep enough copies in flight
// and the arithmetic out of their way.
//
// A CTA holds a ring of tiles of 64 keys and values that one warp fills with
// TMA (128-byte swizzle, one box per page and 64 columns).  RG groups of four
// warps own 8 query rows each; a group's warps take 16 keys of every tile
// each, with their own m, l and O, and join them through shared memory at the
// end of an item.  The products run on the warp-level tensor instructions
// (m16n8k16): 16 rows are too few for tensor memory's 128.
//
// Precision: keys and values enter as stored.  Each fp32 query is split in two
// 16-bit numbers (split16) and the two parts of 8 rows make up the
// instruction's 16 rows -- rows 0-7 the rounded queries, rows 8-15 what the
// rounding left -- so that the split costs nothing; the sums of both halves
// are added in fp32.  The probabilities are split the same way.
#include "paged.cuh"

#include <algorithm>
#include <mutex>

namespace sq {
namespace {

constexpr int kKT = 64;      // keys per tile
constexpr int kItems = 4;    // pieces the producer may be ahead
constexpr int kMinPairs = 2; // key tiles of a CTA's share at least

template <int D, int RG>
struct RowsCfg {
    static constexpr int kThreads = RG * 128 + 32;
    static constexpr int kTileBytes = kKT * D * 2;  // keys, or values, of a tile
    static constexpr int kStages = (RG == 1 ? 196608 : 163840) / (2 * kTileBytes);
    static constexpr int kJoin = RG * 4 * 8 * D * 4;  // [group][warp][row][D] outputs
    static constexpr int kSmem = kStages * 2 * kTileBytes + kJoin + 1024;
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

template <int D, bool BF, int RG>
__global__ void __launch_bounds__(RowsCfg<D, RG>::kThreads, 1)
    paged_rows_kernel(const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV, const __grid_constant__ PagedArgs a,
                      int bx) {
    using C = RowsCfg<D, RG>;
    constexpr int ST = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float *join = reinterpret_cast<float *>(smem + ST * 2 * C::kTileBytes);
    __shared__ uint64_t full[ST], empty[ST], item_full[kItems], item_empty[kItems], grp[RG];
    __shared__ unsigned char holes[ST];  // bit i: the i-th box of the tile's keys is missing
    __shared__ Piece items[kItems];
    __shared__ Share share;
    __shared__ float2 join_ml[RG][4][8];
    __shared__ int last_flag[RG];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &abort_flag;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            bar_init(&full[i], 1);
            bar_init(&empty[i], RG * 4);
        }
        for (int i = 0; i < kItems; ++i) {
            bar_init(&item_full[i], 1);
            bar_init(&item_empty[i], RG * 4);
        }
        for (int i = 0; i < RG; ++i) bar_init(&grp[i], 4);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();  // every global-memory access below follows the previous kernel
    find_share<kKT, C::kThreads>(a, kMinPairs, &share);

    if (warp == RG * 4) {
        // ------------------------------------------------------------ copies
        const uint32_t sbase = su32(smem);
        const int nsub = kKT / bx;  // boxes along the tile's keys
        const int page_rows = 1 << a.page_shift;
        const int rows_total = a.num_pages * a.Hkv << a.page_shift;
        Walk<kKT> walk;
        walk.start(a, share);
        uint32_t tile = 0;  // tiles copied so far
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            Piece p;
            const bool more = walk.next(a, share, p);
            const int slot = n % kItems;
            if (n >= kItems &&
                !warp_wait(&item_empty[slot], (n / kItems - 1) & 1u, abort, a.error))
                break;
            if (lane == 0) {
                if (more) items[slot] = p;
                else items[slot].stop = 1;
                bar_arrive(&item_full[slot]);
            }
            if (!more) break;
            const int *pages = a.prefix_phase ? a.prefix_pages
                                              : a.block_table + (int64_t)p.seq * a.max_pages;
            const int first_key = a.prefix_phase ? 0 : a.prefix_len;
            int held = -1, entry = -1;  // lane i holds the page-table entry 32 held + i
            for (int i = 0; i < p.ntiles; ++i, ++tile) {
                const int st = tile % ST;
                const int key0 = p.key0 + i * kKT;
                // the tile's pages: the entries lane by lane, 32 at a time
                int row = rows_total;  // past the end: the copy brings zeros
                unsigned miss = 0;
                for (int sub = 0; sub < nsub; ++sub) {
                    const int key = key0 + sub * bx;
                    const int idx = key >> a.page_shift;
                    const bool in = key < p.keys && key + bx > first_key;
                    int e = -1;
                    if (in) {
                        if (idx >> 5 != held) {
                            held = idx >> 5;
                            const int at = (held << 5) + lane;
                            entry = (int64_t)at << a.page_shift < p.keys ? __ldg(pages + at) : -1;
                        }
                        e = __shfl_sync(0xffffffffu, entry, idx & 31);
                    }
                    const bool there = e >= 0 && e < a.num_pages;
                    if (!there) miss |= 1u << sub;
                    // lane: sub-box, 64-column slab, keys or values
                    if (there && lane % nsub == sub)
                        row = ((e * a.Hkv + p.head) << a.page_shift) + (key & (page_rows - 1));
                }
                if (tile >= ST && !warp_wait(&empty[st], (tile / ST - 1) & 1u, abort, a.error)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    holes[st] = (unsigned char)miss;
                    bar_expect(&full[st], 2 * C::kTileBytes);
                }
                __syncwarp();
                if (lane < nsub * (D / 64) * 2) {
                    const int sub = lane % nsub, rest = lane / nsub;
                    const int slab = rest % (D / 64), kv = rest / (D / 64);
                    tma_box(sbase + (2 * st + kv) * C::kTileBytes + slab * kKT * 128 +
                                sub * bx * 128,
                            kv ? &mapV : &mapK, &full[st], slab * 64, row);
                }
            }
        }
        // every copy issued has landed before the shared memory can go away
        if (lane == 0)
            for (uint32_t i = tile > ST ? tile - ST : 0; i < tile; ++i)
                drain_bar(&full[i % ST], (i / ST) & 1u, a.error);
    } else {
        // ------------------------------------------------- products and softmax
        const int rg = warp >> 2, w = warp & 3;
        const int g = lane >> 2, t = lane & 3;  // fragment row and column pair
        const int gt = threadIdx.x & 127;       // thread of the group
        uint32_t gphase = 0;
        // the group's four warps meet (bounded, so that an abort leaves nobody behind)
        auto group_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) bar_arrive(&grp[rg]);
            const bool ok = warp_wait(&grp[rg], gphase & 1u, abort, a.error);
            ++gphase;
            return ok;
        };
        uint32_t tile = 0;
        for (uint32_t n = 0;; ++n) {
            const int slot = n % kItems;
            if (!warp_wait(&item_full[slot], (n / kItems) & 1u, abort, a.error)) break;
            const Piece p = items[slot];
            __syncwarp();
            if (lane == 0) bar_arrive(&item_empty[slot]);
            if (p.stop) break;
            const int row = rg * 8 + g;  // this thread's row of the item
            const int tok = row / a.G;
            const bool live = tok < p.ntok;
            const int limit = live ? row_limit(a, p, tok) : p.keys;
            const int first_key = a.prefix_phase ? 0 : a.prefix_len;
            // the queries, split: a0, a2 rounded (rows 0-7), a1, a3 the rest (rows 8-15)
            uint32_t qf[D / 16][4];
            const float *qrow = a.Q + (int64_t)(p.tok0 + tok) * a.ldq +
                                (p.head * a.G + row % a.G) * D;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                float2 x = make_float2(0.f, 0.f), y = x;
                if (live) {
                    x = *reinterpret_cast<const float2 *>(qrow + 16 * i + 2 * t);
                    y = *reinterpret_cast<const float2 *>(qrow + 16 * i + 2 * t + 8);
                }
                split16<BF>(x.x * a.sign, x.y * a.sign, qf[i][0], qf[i][1]);
                split16<BF>(y.x * a.sign, y.y * a.sign, qf[i][2], qf[i][3]);
            }
            float o[D / 8][4];
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int it = 0; it < p.ntiles; ++it, ++tile) {
                const int st = tile % ST;
                if (!warp_wait(&full[st], (tile / ST) & 1u, abort, a.error)) {
                    ok = false;
                    break;
                }
                const uint32_t ks = su32(smem) + 2 * st * C::kTileBytes;
                const uint32_t vs = ks + C::kTileBytes;
                const int key0 = p.key0 + it * kKT + 16 * w;  // this warp's keys
                // logits of 8 rows x 16 keys, both halves of the split
                float s[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
                {
                    const int kr = 16 * w + (lane >> 4) * 8 + (lane & 7);
                    const uint32_t base = ks + kr * 128;
                    const int half = (lane >> 3) & 1;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t b[4];
                        ldsm4(b, base + (i / 4) * kKT * 128 +
                                     ((((2 * i + half) & 7) ^ (kr & 7)) << 4));
                        mma16816<BF>(s[0], qf[i], b[0], b[1]);
                        mma16816<BF>(s[1], qf[i], b[2], b[3]);
                    }
                }
                float x[4] = {s[0][0] + s[0][2], s[0][1] + s[0][3], s[1][0] + s[1][2],
                              s[1][1] + s[1][3]};
                const bool missing = (holes[st] >> (16 * w / bx)) & 1;
                // does the mask cut this warp's keys?
                const bool cut = key0 + 16 > p.keys || key0 < first_key || missing;
                uint32_t vmask0 = 0xffffffffu, vmask1 = 0xffffffffu;
                if (__any_sync(0xffffffffu, cut || key0 + 16 > limit)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + 8 * (i >> 1) + 2 * t + (i & 1);
                        if (missing || key >= limit || key < first_key) x[i] = -INFINITY;
                    }
                    // rows of the tile that hold no key of the sequence may hold
                    // anything: their values are taken as zeros
                    auto there = [&](int key) {
                        return key < p.keys && key >= first_key ? 0xffffu : 0u;
                    };
                    vmask0 = there(key0 + 2 * t) | there(key0 + 2 * t + 1) << 16;
                    vmask1 = there(key0 + 2 * t + 8) | there(key0 + 2 * t + 9) << 16;
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = mx == -INFINITY ? m : fmaxf(m, mx * a.scale);
                if (__any_sync(0xffffffffu, mn > m)) {
                    const float f = max_factor(m, mn);
                    l *= f;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        o[i][0] *= f;
                        o[i][1] *= f;
                        o[i][2] *= f;
                        o[i][3] *= f;
                    }
                    m = mn;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = x[i] == -INFINITY ? 0.0f : ex2(fmaf(x[i], a.scale, -m));
                    l += x[i];
                }
                uint32_t pf[4];  // a0 / a1: keys 2t, 2t+1 rounded / rest; a2 / a3: keys + 8
                split16<BF>(x[0], x[1], pf[0], pf[1]);
                split16<BF>(x[2], x[3], pf[2], pf[3]);
                {
                    const int kr = 16 * w + ((lane >> 3) & 1) * 8 + (lane & 7);
                    const uint32_t base = vs + kr * 128;
                    const int half = lane >> 4;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t b[4];
                        ldsm4t(b, base + (i / 4) * kKT * 128 +
                                      ((((2 * i + half) & 7) ^ (kr & 7)) << 4));
                        mma16816<BF>(o[2 * i], pf, b[0] & vmask0, b[1] & vmask1);
                        mma16816<BF>(o[2 * i + 1], pf, b[2] & vmask0, b[3] & vmask1);
                    }
                }
                __syncwarp();
                if (lane == 0) bar_arrive(&empty[st]);
            }
            if (!ok) break;
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            // the four warps' results
            float *mine = join + ((rg * 4 + w) * 8 + g) * D;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(mine + 8 * i + 2 * t) =
                    make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3]);
            if (t == 0) join_ml[rg][w][g] = make_float2(m, l);
            if (!group_sync()) break;
            // thread: row gt / 16, D / 16 columns
            constexpr int N = D / 16;
            const int jr = gt >> 4, jc = (gt & 15) * N;
            const int irow = rg * 8 + jr;
            const bool jlive = irow / a.G < p.ntok;
            float jm = -INFINITY, jl = 0.0f, jo[N];
#pragma unroll
            for (int i = 0; i < N; ++i) jo[i] = 0.0f;
            for (int v = 0; v < 4; ++v) jm = fmaxf(jm, join_ml[rg][v][jr].x);
            for (int v = 0; v < 4; ++v) {
                const float2 e = join_ml[rg][v][jr];
                const float f = max_factor(e.x, jm);
                jl += e.y * f;
                const float *src = join + ((rg * 4 + v) * 8 + jr) * D + jc;
#pragma unroll
                for (int i = 0; i < N; ++i) jo[i] += src[i] * f;
            }
            bool write = true;
            if (p.npieces > 1) {
                // this CTA's part of the item, then whoever is last joins them all
                const int64_t base = ((int64_t)(2 * blockIdx.x + p.slot) * RG * 8 + irow);
                float4 *d = reinterpret_cast<float4 *>(a.part_o + base * D + jc);
#pragma unroll
                for (int i = 0; i < N / 4; ++i)
                    __stcg(d + i, make_float4(jo[4 * i], jo[4 * i + 1], jo[4 * i + 2],
                                              jo[4 * i + 3]));
                if (jc == 0) __stcg(a.part_ml + base, make_float2(jm, jl));
                __threadfence();
                if (!group_sync()) break;
                unsigned *count = a.counters + p.first_cta * RG + rg;
                if (gt == 0) {
                    const bool last = atomicAdd(count, 1u) == (unsigned)p.npieces - 1;
                    if (last) *count = 0;  // as the next launch wants it
                    last_flag[rg] = last;
                }
                if (!group_sync()) break;
                write = last_flag[rg] != 0;
                if (write) {
                    __threadfence();
                    jm = -INFINITY;
                    jl = 0.0f;
#pragma unroll
                    for (int i = 0; i < N; ++i) jo[i] = 0.0f;
                    for (int c = 0; c < p.npieces; ++c) {
                        const int64_t from =
                            (int64_t)(2 * (p.first_cta + c) + (c == 0)) * RG * 8 + irow;
                        const float2 e = __ldcg(a.part_ml + from);
                        const float top = fmaxf(jm, e.x);
                        const float f = max_factor(jm, top), fe = max_factor(e.x, top);
                        jm = top;
                        jl = jl * f + e.y * fe;
                        const float4 *src =
                            reinterpret_cast<const float4 *>(a.part_o + from * D + jc);
#pragma unroll
                        for (int i = 0; i < N / 4; ++i) {
                            const float4 v = __ldcg(src + i);
                            jo[4 * i] = jo[4 * i] * f + v.x * fe;
                            jo[4 * i + 1] = jo[4 * i + 1] * f + v.y * fe;
                            jo[4 * i + 2] = jo[4 * i + 2] * f + v.z * fe;
                            jo[4 * i + 3] = jo[4 * i + 3] * f + v.w * fe;
                        }
                    }
                }
            }
            if (write && jlive)
                write_row<D, N>(a,
                                (int64_t)(p.tok0 + irow / a.G) * a.Hq + p.head * a.G + irow % a.G,
                                jc, jm, jl, jo);
            // the buffers are free for the next item
            if (!group_sync()) break;
        }
    }
    __syncthreads();
}

template <int D, bool BF, int RG>
sq_status launch_rows(const PagedArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, int bx,
                      int sms, cudaStream_t st) {
    using C = RowsCfg<D, RG>;
    static std::mutex mu;
    static bool done[64] = {};
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[di.device & 63]) {
            if (cudaFuncSetAttribute(paged_rows_kernel<D, BF, RG>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::kSmem) != cudaSuccess)
                return SQ_ERR_CUDA;
            done[di.device & 63] = true;
        }
    }
    return launch_pdl(paged_rows_kernel<D, BF, RG>, dim3((unsigned)sms), dim3(C::kThreads),
                      C::kSmem, st, 1, mk, mv, a, bx);
}

}  // namespace

sq_status launch_paged_rows(const PagedArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                            int D, bool bf16, int row_groups, int bx, int sms, cudaStream_t st) {
    const int v = (D == 128 ? 4 : 0) + (bf16 ? 2 : 0) + (row_groups == 2 ? 1 : 0);
    switch (v) {
    case 0: return launch_rows<64, false, 1>(a, mk, mv, bx, sms, st);
    case 1: return launch_rows<64, false, 2>(a, mk, mv, bx, sms, st);
    case 2: return launch_rows<64, true, 1>(a, mk, mv, bx, sms, st);
    case 3: return launch_rows<64, true, 2>(a, mk, mv, bx, sms, st);
    case 4: return launch_rows<128, false, 1>(a, mk, mv, bx, sms, st);
    case 5: return launch_rows<128, false, 2>(a, mk, mv, bx, sms, st);
    case 6: return launch_rows<128, true, 1>(a, mk, mv, bx, sms, st);
    default: return launch_rows<128, true, 2>(a, mk, mv, bx, sms, st);
    }
}

}  // namespace sq
