// Attention over the paged cache for many query rows per key/value head, on the
// 5th-generation tensor cores (tcgen05): prompts, chunks of prompts, drafts of
// many heads, and the prefix that a batch shares.
//
// An item is up to 128 query rows (tokens x heads of a group, the instruction's
// M) of one sequence and key/value head; its keys come in tiles of 128.  Per
// tile: S = Q K^T into tensor memory; the softmax of the tile alone, two threads
// per row, whose probabilities take S's place; P V into a second area of tensor
// memory; and from there into the output in registers,
//   O = O 2^(M - M') + (P V) 2^(m - M'),   M' = max(M, m),
// m the tile's row maximum, M the output's.  Since a tile's softmax knows
// nothing of the tiles before it, all four steps run at once on different
// tiles: the products of tile t + 1 and t - 1, the softmax of tile t, the sum of
// tile t - 2, and across items too.  The sum is formed outside the tensor cores,
// whose accumulator truncates: kept there over the 64 tiles of 8192 keys it
// would be off by 6e-6.
//
// Precision.  Keys and values enter as stored; fp32 queries and probabilities
// are split in 16-bit numbers of their type, one instruction per part: two for
// fp16 (within 2^-22), three for bf16 (exact; two would leave 2^-17).
// The probabilities of a tile carry a factor 2^12, and fp16 queries are scaled
// row by row by a power of two, so that no part falls below fp16's range.  The
// queries carry the scale's significand, so that logits are multiplied by a power
// of two: the exponents of a row whose logits are far from one are exact too.
//
// Bound: the products, at twice (fp16) or three times (bf16) the instructions
// of the plain operands' attention, for long items (152 of 16,384 keys, bf16:
// 330 us, 1.48 PFLOP/s of the parts' products, 77 % of the measured bf16 rate);
// for fp16 as much by memory (245 us, 5.2 TB/s).  Short items are bound by their
// start and end: 7 to 9 us for queries, the first products and the rows' way out,
// during which the code of the item's ends comes from memory more often than it
// runs (an instruction that is not in the cache costs about 20 cycles), and
// another 5 us where an item is split and joined.
// Measured: two prompts of about 4000 tokens, 32 / 8 heads of 128, bf16: 717 us
// (the same in fp16 532); 16 drafts of 2 to 5 tokens behind 4096 to 16,384 keys,
// 24 / 4 heads, fp16: 94 us, 57 % of the measured copy rate.  TMA boxes of one
// 16-row page each measured 3.0 TB/s (104 ns of its unit's time a box); cp.async
// 7 TB/s.
//
// Roles (640 threads, one persistent CTA per SM):
//   warps 0-3, 4-7   queries and softmax, 64 keys of a tile each;
//   warps 8-11       the output: sum over the tiles, partial results, rows;
//   warps 12-15      copies: keys and values with cp.async into a ring of
//                    128-row slots in the operands' layout (128-byte swizzle;
//                    rows of no key are zeros);
//   warp 16          tensor memory, and lane 0 issues the products;
//   warp 17          walks the CTA's share and hands its pieces to the others.
// Tensor memory, 512 columns: two areas of 64 columns per part for S and then P,
// and two areas (bf16: one) of 128 for P V.
// Every wait is bounded (4 s); on expiry the CTA records an error for
// sq_device_status, lets its copies and products land and exits.
#include "paged.cuh"

#include <algorithm>
#include <mutex>

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
// Bounded wait for the phase of parity `parity`; false when the CTA aborted.
// (Short, because it is inlined: the registers are split by role, which leaves no
// room for calls.)
__device__ __forceinline__ bool wait_bar(const uint64_t *bar, uint32_t parity,
                                         volatile int *abort, unsigned *error) {
    const uint32_t a = su32(bar);
    if (try_wait(a, parity)) return true;
    const uint64_t t0 = gtime();
#pragma unroll 1
    while (!try_wait(a, parity)) {
        if (*abort) return false;
        if (gtime() - t0 > kPagedTimeoutNs) {
            *abort = 1;
            atomicOr(error, 1u);
            return false;
        }
    }
    return true;
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

constexpr int kKT = 128;     // keys per tile
constexpr int kRows = 128;   // query rows per item
constexpr int kThreads = 640;
constexpr int kItems = 4;    // pieces the walk may be ahead
constexpr int kStats = 4;    // tiles whose maxima and sums are kept
constexpr int kMiss = 8;     // more than the tiles between a copy and its softmax
// Pieces of an item that are joined in one go (2.3 us each; 3 to 12 measured alike;
// all in one go: 322 against 57 us for 8 tokens of 16 heads behind 30,000 keys)
constexpr int kJoin = 6;
// A CTA's share at least, in pairs: 1, 4, 6 and 10 measured 27, 21, 21 and 20 us
// (300 keys, 1 item), 35, 31, 36 and 42 (1024 keys, 19 items), 71, 57, 58 and 62
// (30,000 keys, 1 item)
constexpr int kMinTiles = 4;
constexpr float kBias = 12.0f;  // log2 of the probabilities' factor

template <int D, bool BF>
struct TilesCfg {
    static constexpr int kParts = BF ? 3 : 2;
    static constexpr int kSlab = kKT * 128;            // 128 rows x 64 elements
    static constexpr int kSlot = kSlab * (D / 64);     // keys or values of a tile
    static constexpr int kSlots = D == 64 ? 6 : BF ? 3 : 4;
    static constexpr int kQPart = kRows * D * 2;       // one part of the queries
    static constexpr int kSmem = kParts * kQPart + kSlots * kSlot + 1024;
    // tensor memory: S and P of a tile, S's first column in it, P V
    static constexpr int kArea = 64 * kParts;
    static constexpr int kS0 = kArea - 128;
    // an item's start and end in key tiles (bf16: 2, 4, 6, 8 measured 755, 692,
    // 708, 735 us for two prompts of 4096 tokens; fp16: 672, 534, 506, 528)
    static constexpr int kPad = BF ? 4 : 6;
    static constexpr int kPVs = BF ? 1 : 2;
    static constexpr int kPV0 = 2 * kArea;
};

struct TileBars {
    uint64_t full[6], empty[6];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t q_full, q_empty, s_full[2], p_full[2], pv_full[2], pv_empty[2];
    uint64_t group, pair[4], mma_done;
    uint32_t tmem;
    int abort_flag;
    int last;
    unsigned miss[kMiss];  // bit i: keys 16 i .. 16 i + 15 of the tile are of a missing page
    Piece items[kItems];
    int stop[kItems];
    int bad_from[kItems], bad_to[kItems];  // the tiles (of the share) of a piece that values
                                           // which are not finite were taken out of
    Share share;
    float2 stat[kStats][2][kRows];  // a tile's row maxima (log2 units) and half sums
    float half_max[2][2][kRows];    // a tile's row maxima over its halves
    float qmul[2][kRows];           // what the rows' queries were divided by
};

__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// shared-memory operand, 128-byte swizzle: 8-row atoms of 1024 bytes.  The
// descriptor's low word: the address in 16-byte units and `lead`, the distance of
// 64-element groups of an operand that is not K-major; its high word is constant.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lead) {
    return (saddr & 0x3FFFFu) >> 4 | (lead >> 4) << 16;
}
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
// kind::f16: fp32 sums of bf16 or fp16 operands, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool bf16, bool b_by_rows) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_by_rows ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}
// A from tensor memory: 8 columns hold K = 16
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            su32(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ PagedArgs a, const uint16_t *__restrict__ k_cache,
                       const uint16_t *__restrict__ v_cache) {
    using C = TilesCfg<D, BF>;
    constexpr int NS = C::kSlots, NP = C::kParts;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ TileBars B;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &B.abort_flag;
    const uint32_t qbase = su32(smem);  // [part][slab][128 rows][128 B]
    const uint32_t ring = qbase + NP * C::kQPart;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            bar_init(&B.full[i], 4);
            bar_init(&B.empty[i], 1);
        }
        for (int i = 0; i < kItems; ++i) {
            bar_init(&B.item_full[i], 1);
            bar_init(&B.item_empty[i], 17);
        }
        bar_init(&B.q_full, 8);
        bar_init(&B.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&B.s_full[i], 1);
            bar_init(&B.p_full[i], 8);
            bar_init(&B.pv_full[i], 1);
            bar_init(&B.pv_empty[i], 4);
        }
        bar_init(&B.group, 4);
        for (int i = 0; i < 4; ++i) bar_init(&B.pair[i], 2);
        bar_init(&B.mma_done, 1);
        for (int i = 0; i < kItems; ++i) {
            B.bad_from[i] = 0x7fffffff;
            B.bad_to[i] = -1;
        }
        B.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         su32(&B.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    pdl_wait();  // every global-memory access below follows the previous kernel
    pdl_launch_dependents();  // (after it: see begin_rows)
    find_shares<kKT, C::kPad, kThreads, 1>(a, kMinTiles, &B.share);
    const uint32_t tmem = B.tmem;

    // registers: 96 a thread at launch; (2 x 104 + 168 + 56 + 48) x 128 in all
    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 16 && lane == 0) {
            // ------------------------------------------------------ products
            // per tile t of the share: S(t + 1) is issued before P V(t)
            const uint32_t qk_desc = idesc_f16(kKT, BF, false), pv_desc = idesc_f16(D, BF, true);
            uint32_t item = 0;        // pieces begun
            int left = 0;             // tiles of the piece still without S
            uint32_t t_s = 0, t_pv = 0;  // tiles with S, with P V issued
            // slots in the copies' order: K0, then K(t + 1), V(t), ..., the last V
            bool ok = true, more = true;
            auto next_s = [&]() {
                if (left == 0) {
                    const int it = item % kItems;
                    ok = wait_bar(&B.item_full[it], (item / kItems) & 1u, abort, a.error);
                    if (!ok) return;
                    more = !B.stop[it];
                    if (!more) return;
                    left = B.items[it].ntiles;
                    bar_arrive(&B.item_empty[it]);
                    ok = wait_bar(&B.q_full, item & 1u, abort, a.error);
                    if (!ok) return;
                    ++item;
                }
                const uint32_t ks = t_s == 0 ? 0 : 2 * t_s - 1;
                ok = wait_bar(&B.full[ks % NS], (ks / NS) & 1u, abort, a.error);
                if (!ok) return;
                tc_after();
                const uint32_t kb = ring + (ks % NS) * C::kSlot;
                const uint32_t d = tmem + (t_s & 1) * C::kArea + C::kS0;
                // the smallest part first: what the accumulator truncates is relative
                // to the sum so far
                const uint32_t qd = desc_low(qbase, 16), kd = desc_low(kb, 16);
#pragma unroll
                for (int part = NP - 1; part >= 0; --part)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int step = (i / 4) * C::kSlab / 16 + 2 * (i % 4);
                        mma_ss(d, qd + part * C::kQPart / 16 + step, kd + step, qk_desc,
                               (part < NP - 1 || i) ? 1u : 0u);
                    }
                if (--left == 0) mma_commit(&B.q_empty);  // (before the softmax can go on)
                mma_commit(&B.s_full[t_s & 1]);
                mma_commit(&B.empty[ks % NS]);
                ++t_s;
            };
            while (ok) {
                if (more) next_s();
                if (!ok) break;
                if (more && t_s - t_pv < 2) continue;  // the first tile
                if (t_pv == t_s) break;
                // the last tile's values follow their keys at once
                const uint32_t vs = t_pv + 1 < t_s ? 2 * t_pv + 2 : 2 * t_pv + 1;
                const uint32_t pb = t_pv % C::kPVs;
                ok = wait_bar(&B.full[vs % NS], (vs / NS) & 1u, abort, a.error) &&
                     wait_bar(&B.p_full[t_pv & 1], (t_pv >> 1) & 1u, abort, a.error) &&
                     (t_pv < C::kPVs || wait_bar(&B.pv_empty[pb], (t_pv / C::kPVs - 1) & 1u,
                                                 abort, a.error));
                if (!ok) break;
                tc_after();
                const uint32_t d = tmem + C::kPV0 + 128 * pb;
                const uint32_t pa = tmem + (t_pv & 1) * C::kArea;
                const uint32_t v = ring + (vs % NS) * C::kSlot;
                const uint32_t vd = desc_low(v, C::kSlab);
#pragma unroll
                for (int part = NP - 1; part >= 0; --part)
#pragma unroll
                    for (int i = 0; i < kKT / 16; ++i)
                        mma_ts(d, pa + 8 * NP * i + 8 * part, vd + 128 * i, pv_desc,
                               (part < NP - 1 || i) ? 1u : 0u);
                mma_commit(&B.pv_full[pb]);
                mma_commit(&B.empty[vs % NS]);
                ++t_pv;
            }
            // every product issued completes before tensor memory is freed
            mma_commit(&B.mma_done);
            drain_bar(&B.mma_done, 0, a.error);
        } else if (warp == 17) {
            // -------------------------------------------- the share's pieces
            Walk<kKT, C::kPad> walk;
            walk.start(a, B.share);
            for (uint32_t n = 0;; ++n) {
                Piece p;
                const bool more = walk.next(a, B.share, p);
                const int it = n % kItems;
                if (n >= kItems &&
                    !warp_wait(&B.item_empty[it], (n / kItems - 1) & 1u, abort, a.error))
                    break;
                if (more && a.prefix_phase) {
                    // what every row sees: of the prefix, the least that any does
                    int least = a.prefix_len;
                    for (int i = lane; i < p.ntok; i += 32) least = min(least, row_limit(a, p, i));
                    p.pos0 = __reduce_min_sync(0xffffffffu, least) - 1;
                }
                if (lane == 0) {
                    B.stop[it] = !more;
                    if (more) B.items[it] = p;
                    bar_arrive(&B.item_full[it]);
                }
                __syncwarp();
                if (!more) break;
            }
        }
        __syncwarp();
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // ------------------------------------------------------------ copies
        const int ct = threadIdx.x - 384;
        uint32_t seq = 0, done = 0, tile = 0;  // slots begun, slots handed over, tiles begun
        bool ok = true;
        // thread: chunk ch of rows r0, r0 + kRowStep, ... of a slot
        constexpr int kRowStep = 128 / (D / 8);
        const int r0 = ct / (D / 8), ch = ct % (D / 8);
        const uint32_t my_chunk =
            (ch >> 3) * C::kSlab + r0 * 128 + (((ch & 7) ^ (r0 & 7)) << 4);
        uint32_t scan = 0;  // 4 bits per slot: 1 + the piece's slot where values are looked at
        auto hand_over = [&](bool all) {
            if (all) asm volatile("cp.async.wait_group 0;" ::: "memory");
            else asm volatile("cp.async.wait_group 1;" ::: "memory");
            if (scan != 0) {
                // A masked key's probability is zero, but its value need not be
                // finite, and zero times that is NaN: in tiles of which a row does not
                // see every key such values are taken out here (each thread its own
                // copies) and left to the item's end.  (In the other tiles they stay in
                // the product: every row sees them, and none of its sum is finite.)
                for (uint32_t d = done; d < seq - (all ? 0 : 1); ++d) {
                    const int s4 = 4 * (d % NS);
                    const uint32_t who = scan >> s4 & 15u;
                    if (who == 0) continue;
                    scan &= ~(15u << s4);
                    const uint32_t from = ring + (d % NS) * C::kSlot + my_chunk;
                    uint32_t bad = 0;
#pragma unroll 4
                    for (int j = 0; j < kKT / kRowStep; ++j) {
                        uint32_t w[4];
                        lds4(w, from + j * kRowStep * 128);
                        bad |= not_finite<BF>(w[0]) | not_finite<BF>(w[1]) |
                               not_finite<BF>(w[2]) | not_finite<BF>(w[3]);
                    }
                    if (bad) {
                        const int t = (int)(d - 1) / 2;  // the tile whose values slot d holds
                        atomicMin(&B.bad_from[who - 1], t);
                        atomicMax(&B.bad_to[who - 1], t);
#pragma unroll 1
                        for (int j = 0; j < 4 * (kKT / kRowStep); ++j) {
                            const uint32_t at = from + (j >> 2) * kRowStep * 128 + 4 * (j & 3);
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at),
                                         "r"(finite_part<BF>(w))
                                         : "memory");
                        }
                    }
                }
            }
            fence_async_smem();
            __syncwarp();
            while (done < seq - (all ? 0 : 1)) {
                if (lane == 0) bar_arrive(&B.full[done % NS]);
                ++done;
            }
        };
        // 128 rows of a cache into the next slot; lane l (of 8) holds the place of
        // rows 16 l .. 16 l + 15 in the caches, in bytes
        auto copy_slot = [&](const uint16_t *cache, int64_t place, unsigned miss, int lo, int hi,
                             uint32_t look) {
            const uint32_t sl = seq % NS;
            if (seq >= NS) {
                const uint32_t ph = (seq / NS - 1) & 1u;
                // no free slot yet: what has been copied is handed over first
                if (done < seq && !__all_sync(0xffffffffu, try_wait(su32(&B.empty[sl]), ph)))
                    hand_over(true);
                if (!warp_wait(&B.empty[sl], ph, abort, a.error)) {
                    ok = false;
                    return;
                }
            }
            const uint32_t dst = ring + sl * C::kSlot + my_chunk;
            scan |= look << 4 * sl;
            const char *src = reinterpret_cast<const char *>(cache) + (r0 * D + ch * 8) * 2;
            if (miss == 0 && lo <= 0 && hi >= kKT) {
#pragma unroll
                for (int j = 0; j < kKT / 16; ++j) {
                    const char *from = src + __shfl_sync(0xffffffffu, place, j);
#pragma unroll
                    for (int i = 0; i < 16 / kRowStep; ++i)
                        copy16(dst + (16 * j + i * kRowStep) * 128, from + i * kRowStep * D * 2, true);
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < kKT / 16; ++j) {
                    const char *from = src + __shfl_sync(0xffffffffu, place, j);
                    const bool page = !(miss >> j & 1);
#pragma unroll
                    for (int i = 0; i < 16 / kRowStep; ++i) {
                        const int r = 16 * j + r0 + i * kRowStep;
                        const bool in = page && r < hi && r >= lo;
                        copy16(dst + (16 * j + i * kRowStep) * 128,
                               in ? from + i * kRowStep * D * 2
                                  : reinterpret_cast<const char *>(cache),
                               in);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++seq;
            if (seq - done > 1) hand_over(false);
        };
        // a turn copies the keys of tile `tile` and the values of the one before;
        // the last turn the last values alone
        int64_t v_place = 0;
        unsigned v_miss = 0;
        int v_lo = 0, v_hi = 0, left = 0, key0 = 0;
        uint32_t v_look = 0;
        Piece p = {};
        bool more = true;
        int entry = -1;
        // lane l: the entry of the page of keys 16 (l % 8) .. of a tile; -1 where none is
        // wanted
        auto page_of = [&](const KeyRange &r) {
            const int *pages = r.front ? a.prefix_pages
                                       : a.block_table + (int64_t)p.seq * a.max_pages;
            const int key = r.key + 16 * (lane & 7);
            return key < r.hi && key + 16 > r.lo ? __ldg(pages + (key >> a.page_shift)) : -1;
        };
        for (uint32_t n = 0; ok && more;) {
            if (left == 0) {
                const int it = n % kItems;
                if (!warp_wait(&B.item_full[it], (n / kItems) & 1u, abort, a.error)) {
                    ok = false;
                    break;
                }
                more = !B.stop[it];
                if (more) {
                    p = B.items[it];
                    left = p.ntiles;
                    key0 = p.key0;
                    entry = page_of(key_range(a, key0, p.keys));
                    __syncwarp();
                    if (lane == 0) bar_arrive(&B.item_empty[it]);
                    ++n;
                }
            }
            int64_t place = 0;
            unsigned miss = 0;
            int lo = 0, hi = 0;
            uint32_t look = 0;
            if (more) {
                // the next tile's entry is on its way meanwhile
                const int e = entry;
                const KeyRange r = key_range(a, key0, p.keys);
                const int key = r.key + 16 * (lane & 7);
                lo = r.lo - r.key;
                hi = r.hi - r.key;
                if (key_range(a, key0, p.pos0 + 1).hi < r.key + kKT)
                    look = 1 + (n - 1) % kItems;  // (the piece's first row does not see all)
                entry = left > 1 ? page_of(key_range(a, key0 + kKT, p.keys)) : -1;
                const bool there = e >= 0 && e < a.num_pages;
                miss = ~__ballot_sync(0xffffffffu, there) & 0xffu;
                if (there)
                    place = ((((int64_t)e * a.Hkv + p.head) << a.page_shift) +
                             (key & ((1 << a.page_shift) - 1))) *
                            (D * 2);
                if (ct == 0) B.miss[tile % kMiss] = miss;
            }
#pragma unroll 1
            for (int kv = more ? 0 : 1; kv < (tile > 0 ? 2 : 1) && ok; ++kv)
                copy_slot(kv ? v_cache : k_cache, kv ? v_place : place, kv ? v_miss : miss,
                          kv ? v_lo : lo, kv ? v_hi : hi, kv ? v_look : 0u);
            v_place = place;
            v_miss = miss;
            v_lo = lo;
            v_hi = hi;
            v_look = look;
            if (more) {
                ++tile;
                --left;
                key0 += kKT;
            }
        }
        if (ok && done < seq) hand_over(true);
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // ---------------------------------------------- queries and softmax
        const int g = warp >> 2, w = warp & 3;
        const int r = 32 * w + lane;  // row of the item, tensor-memory lane
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
        uint32_t t = 0;  // tiles of the share so far
        for (uint32_t n = 0;; ++n) {
            const int it = n % kItems;
            if (!warp_wait(&B.item_full[it], (n / kItems) & 1u, abort, a.error)) break;
            if (B.stop[it]) break;
            const Piece &p = B.items[it];  // held until the piece is done
            {
                // 16 rows of the queries, a row (D = 64: two) per step: copied as they
                // are into the place of their parts, then split there.  (Short loops:
                // this runs once an item, and an instruction that is not in the cache
                // costs more than it saves; unrolled, with the rows in registers, it
                // took 7800 cycles.)
                constexpr int LPR = D / 4;      // lanes per row
                constexpr int RPS = 32 / LPR;   // rows per step
                const int sub = lane / LPR, c4 = lane % LPR;
                const int part4 = c4 / (D / 8), in4 = c4 % (D / 8);
                // lane l (of 16) knows where row l is
                const int lr = 16 * warp + (lane & 15), lt = lr * a.g_inv >> 16;
                int64_t place = -1;
                if (lt < p.ntok)
                    place = (int64_t)(p.tok0 + lt) * a.ldq + (p.head * a.G + (lr - lt * a.G)) * D;
                // the piece before has no S to be formed any more
                if (n > 0 && !warp_wait(&B.q_empty, (n - 1) & 1u, abort, a.error)) break;
                const uint32_t rows = qbase + (16 * warp + sub) * 128;
                const uint32_t raw = rows + part4 * C::kQPart + (in4 >> 3) * C::kSlab;
                const uint32_t to = rows + (c4 >> 4) * C::kSlab + (c4 & 1) * 8;
#pragma unroll 2
                for (int i = 0; i < 16; i += RPS) {
                    const int64_t at = __shfl_sync(0xffffffffu, place, i + sub);
                    copy16(raw + i * 128 + (((in4 & 7) ^ ((i + sub) & 7)) << 4),
                           a.Q + (at < 0 ? 0 : at + 4 * c4), at >= 0);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
                for (int i = 0; i < 16; i += RPS) {
                    float4 q;
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w)
                                 : "r"(raw + i * 128 + (((in4 & 7) ^ ((i + sub) & 7)) << 4))
                                 : "memory");
                    float mul = a.q_factor;
                    if (!BF) {
                        // (over the row's own lanes: a step may hold two rows, and what
                        // one of them holds must not cost the other its bits)
                        const float top =
                            fabsf(mul) * fmaxf(fmaxf(fabsf(q.x), fabsf(q.y)),
                                               fmaxf(fabsf(q.z), fabsf(q.w)));
                        unsigned e = __float_as_uint(top);
                        if (LPR == 32) {
                            e = __reduce_max_sync(0xffffffffu, e);
                        } else {
#pragma unroll
                            for (int o = LPR / 2; o > 0; o >>= 1)
                                e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
                        }
                        e >>= 23;
                        const int sh = shift_of((int)e - 127);
                        mul *= pow2(-sh);
                        if (c4 == 0) B.qmul[n & 1][16 * warp + i + sub] = pow2(sh);
                    }
                    uint32_t x[NP], y[NP];
                    split16<BF, NP>(q.x * mul, q.y * mul, x);
                    split16<BF, NP>(q.z * mul, q.w * mul, y);
                    __syncwarp();  // every lane has its numbers of these rows
                    const uint32_t at =
                        to + i * 128 + ((((c4 & 15) >> 1) ^ ((i + sub) & 7)) << 4);
#pragma unroll
                    for (int part = 0; part < NP; ++part)
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at +
                                                                              part * C::kQPart),
                                     "r"(x[part]), "r"(y[part])
                                     : "memory");
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(&B.q_full);
            }
            const int tok = r * a.g_inv >> 16;
            const int limit = tok < p.ntok ? row_limit(a, p, tok) : p.keys;
            int key0 = p.key0;
            bool ok = true;
            for (int k = 0; k < p.ntiles; ++k, ++t, key0 += kKT) {
                const uint32_t area = lanes + (t & 1) * C::kArea;
                if (!warp_wait(&B.s_full[t & 1], (t >> 1) & 1u, abort, a.error)) {
                    ok = false;
                    break;
                }
                tc_after();
                uint32_t v[2][32];
                tmem_ld32(area + C::kS0 + 64 * g, v[0]);
                tmem_ld32(area + C::kS0 + 64 * g + 32, v[1]);
                tmem_ld_wait();
                const unsigned miss = B.miss[t % kMiss] >> (4 * g);
                const float c = BF ? a.scale : a.scale * B.qmul[n & 1][r];
                const KeyRange kr = key_range(a, key0, limit);
                const int at = kr.key + 64 * g;  // this warp's 64 keys
                if (__any_sync(0xffffffffu, at + 64 > kr.hi || at < kr.lo || (miss & 15u) != 0)) {
                    // keys behind the row's own, in front of the suffix or of a
                    // missing page: bit i of `seen` is clear
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int hi = kr.hi - at - 32 * q, lo = kr.lo - at - 32 * q;
                        unsigned seen = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1;
                        if (lo > 0) seen = lo >= 32 ? 0u : seen & (~0u << lo);
                        if (miss >> (2 * q) & 1) seen &= 0xffff0000u;
                        if (miss >> (2 * q + 1) & 1) seen &= 0xffffu;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen >> i & 1)) v[q][i] = 0xff800000u;
                    }
                }
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 64; i += 2)
                    mx = fmaxf(mx, fmaxf(__uint_as_float(v[i / 32][i % 32]),
                                         __uint_as_float(v[i / 32][i % 32 + 1])));
                // the row's maximum, with the other half's; every logit of these
                // rows is in registers from here on
                B.half_max[t & 1][g][r] = mx;
                __syncwarp();
                if (lane == 0) bar_arrive(&B.pair[w]);
                if (!warp_wait(&B.pair[w], t & 1u, abort, a.error)) {
                    ok = false;
                    break;
                }
                mx = fmaxf(mx, B.half_max[t & 1][1 - g][r]);
                // (rounded up: mx c is exact, so the largest exponent is 12 at most, and
                // at least 0 where 12 is less than the maximum's last place)
                const float m = mx == -INFINITY ? 0.0f : __fmaf_ru(mx, c, -kBias);
                const unsigned long long c2 = pk(c, c), m2 = pk(-m, -m);
                unsigned long long sum2 = 0;
                // per 16 keys 8 columns of each part
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t parts[NP][8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = 16 * (q & 1) + 2 * i;
                        float x, y;
                        upk(fma2(pk(__uint_as_float(v[q >> 1][e]),
                                    __uint_as_float(v[q >> 1][e + 1])),
                                 c2, m2),
                            x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sum2 = add2(sum2, pk(x, y));
                        uint32_t z[NP];
                        split16<BF, NP>(x, y, z);
#pragma unroll
                        for (int part = 0; part < NP; ++part) parts[part][i] = z[part];
                    }
#pragma unroll
                    for (int part = 0; part < NP; ++part)
                        tmem_st8(area + 8 * NP * (4 * g + q) + 8 * part, parts[part]);
                }
                float sa, sb;
                upk(sum2, sa, sb);
                B.stat[t % kStats][g][r] = make_float2(mx == -INFINITY ? mx : m, sa + sb);
                tmem_st_wait();
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&B.p_full[t & 1]);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) bar_arrive(&B.item_empty[it]);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        // -------------------------------------------------------- the output
        const int w = warp & 3;
        const int row = 32 * w + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16) + C::kPV0;
        uint32_t t = 0, met = 0;
        // the four warps meet (bounded, so that an abort leaves nobody behind)
        auto group_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) bar_arrive(&B.group);
            return warp_wait(&B.group, met++ & 1u, abort, a.error);
        };
        for (uint32_t n = 0;; ++n) {
            const int it = n % kItems;
            if (!warp_wait(&B.item_full[it], (n / kItems) & 1u, abort, a.error)) break;
            if (B.stop[it]) break;
            const Piece &p = B.items[it];  // held until the piece is done
            unsigned long long o2[D / 2];  // the row's output, in pairs
            float m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 2; ++i) o2[i] = 0;
            const int tok = row * a.g_inv >> 16;
            const bool live = tok < p.ntok;
            const int64_t out =
                live ? (int64_t)(p.tok0 + tok) * a.Hq + p.head * a.G + (row - tok * a.G) : -1;
            if (live && starts_with_prefix(a, p)) {
                const float2 f = __ldcg(a.prefix_ml + out);
                m = f.x;
                l = f.y;
                const ulonglong2 *src =
                    reinterpret_cast<const ulonglong2 *>(a.prefix_o + out * D);
#pragma unroll
                for (int i = 0; i < D / 4; ++i) {
                    const ulonglong2 v = __ldcg(src + i);
                    o2[2 * i] = v.x;
                    o2[2 * i + 1] = v.y;
                }
            }
            bool ok = true;
            for (int k = 0; k < p.ntiles; ++k, ++t) {
                const uint32_t pb = t % C::kPVs;
                if (!warp_wait(&B.pv_full[pb], (t / C::kPVs) & 1u, abort, a.error)) {
                    ok = false;
                    break;
                }
                tc_after();
                float2 e = B.stat[t % kStats][0][row];
                e.y += B.stat[t % kStats][1][row].y;
                const float top = fmaxf(m, e.x);
                const float f = max_factor(m, top), g = max_factor(e.x, top);
                m = top;
                l = l * f + e.y * g;
                const unsigned long long f2 = pk(f, f), g2 = pk(g, g);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t v[16];
                    tmem_ld16(lanes + 128 * pb + 16 * c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o2[8 * c + i] = fma2(pk(__uint_as_float(v[2 * i]),
                                                __uint_as_float(v[2 * i + 1])),
                                             g2, mul2(o2[8 * c + i], f2));
                }
                tc_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&B.pv_empty[pb]);
            }
            if (!ok) break;
            // a row per thread: 32 lines per store, but code that is executed once
            // an item has to be short (an instruction that is not in the cache
            // costs about 20 cycles; rows turned in shared memory measured three
            // times as long)
            const bool whole = p.npieces == 1;
            const int64_t part = (int64_t)(2 * blockIdx.x + p.slot) * kRows + row;
            float *dst = a.part_o + part * D;
            float factor = 1.0f;
            if (whole) {
                factor = row_factor(a, out < 0 ? 0 : out, m, l, live);
                dst = row_target(a) + out * D;
            } else {
                __stcg(a.part_ml + part, make_float2(m, l));
            }
            if (!whole || live) {
                const unsigned long long f2 = pk(factor, factor);
#pragma unroll
                for (int i = 0; i < D / 4; ++i) {
                    float4 v;
                    upk(mul2(o2[2 * i], f2), v.x, v.y);
                    upk(mul2(o2[2 * i + 1], f2), v.z, v.w);
                    __stcg(reinterpret_cast<float4 *>(dst) + i, v);
                }
            }
            if (B.bad_to[it] >= 0) {
                // values that the copies took out of the tiles that not every row sees
                // in full: added to the rows that see them
                float *own = dst;
                if (live) {
                    const int limit = row_limit(a, p, tok);
                    const int t0 = (int)t - p.ntiles;  // the piece's first tile
#pragma unroll 1
                    for (int k = B.bad_from[it] - t0; k <= B.bad_to[it] - t0; ++k) {
                        const int k0 = p.key0 + k * kKT;
                        const KeyRange kr = key_range(a, k0, limit);
                        if (key_range(a, k0, p.pos0 + 1).hi >= kr.key + kKT) continue;
                        const int *pages = kr.front ? a.prefix_pages
                                                    : a.block_table + (int64_t)p.seq * a.max_pages;
                        const int to = min(kr.hi, kr.key + kKT);
#pragma unroll 1
                        for (int key = max(kr.lo, kr.key); key < to; ++key) {
                            const int e = __ldg(pages + (key >> a.page_shift));
                            if (e < 0 || e >= a.num_pages) continue;
                            const uint16_t *v =
                                v_cache + ((((int64_t)e * a.Hkv + p.head) << a.page_shift) +
                                           (key & ((1 << a.page_shift) - 1))) * D;
#pragma unroll 1
                            for (int c = 0; c < D; c += 8) {
                                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(v + c));
                                if (!(not_finite<BF>(x.x) | not_finite<BF>(x.y) |
                                      not_finite<BF>(x.z) | not_finite<BF>(x.w)))
                                    continue;
#pragma unroll 1
                                for (int i = c; i < c + 8; ++i) {
                                    const uint32_t y = v[i];
                                    if (not_finite<BF>(y))
                                        __stcg(own + i, __ldcg(own + i) + widen16<BF>(y));
                                }
                            }
                        }
                    }
                }
                if (!group_sync()) break;
                if (row == 0) {
                    B.bad_from[it] = 0x7fffffff;
                    B.bad_to[it] = -1;
                }
            }
            if (!whole) {
                // this CTA's part of the item is out; whoever is last of a group, and
                // then of the groups, joins them all
                auto from = [&](int c) {  // this warp's rows of piece c
                    return (int64_t)(2 * (p.first + c) + (c == 0)) * kRows + 32 * w;
                };
                const int width = join_width(p.npieces, kJoin);
                Join join = join_of(p, (int)blockIdx.x - p.first, width);
#pragma unroll 1
                for (;;) {
                    __threadfence();
                    if (!(ok = group_sync())) break;
                    if (row == 0) {
                        unsigned *count = a.counters + join.counter;
                        const bool last = atomicAdd(count, 1u) == (unsigned)join.n - 1;
                        if (last) *count = 0;  // as the next launch wants it
                        B.last = last;
                    }
                    if (!(ok = group_sync())) break;
                    if (!B.last) break;  // (rewritten only after the group has met again)
                    __threadfence();
                    m = -INFINITY;
                    for (int c = 0; c < join.n; ++c)
                        m = fmaxf(m, __ldcg(a.part_ml + from(join.first + c * join.step) + lane).x);
                    l = 0.0f;
                    for (int c = 0; c < join.n; ++c) {
                        const float2 e =
                            __ldcg(a.part_ml + from(join.first + c * join.step) + lane);
                        l += e.y * max_factor(e.x, m);
                    }
                    int64_t to = from(join.first) + lane;  // a group's sum: its first piece's place
                    dst = a.part_o;
                    if (join.all) {
                        to = out;
                        factor = row_factor(a, out < 0 ? 0 : out, m, l, live);
                        dst = row_target(a);
                    }
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        // 32 columns of the warp's rows, whole lines
                        float4 sum[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        const int col = 32 * q + 4 * (lane & 7);
#pragma unroll 1
                        for (int c = 0; c < join.n; ++c) {
                            const int64_t piece = from(join.first + c * join.step);
                            const float mc = __ldcg(a.part_ml + piece + lane).x;
                            const float4 *src = reinterpret_cast<const float4 *>(
                                a.part_o + (piece + (lane >> 3)) * D + col);
                            float4 v[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[i] = __ldcg(src + i * D);
                            const float wt = max_factor(mc, m);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float f = __shfl_sync(0xffffffffu, wt, 4 * i + (lane >> 3));
                                sum[i].x += v[i].x * f;
                                sum[i].y += v[i].y * f;
                                sum[i].z += v[i].z * f;
                                sum[i].w += v[i].w * f;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int rr = 4 * i + (lane >> 3);
                            const int64_t to_row = __shfl_sync(0xffffffffu, to, rr);
                            const float f = __shfl_sync(0xffffffffu, factor, rr);
                            if (to_row >= 0)
                                __stcg(reinterpret_cast<float4 *>(dst + to_row * D + col),
                                       make_float4(sum[i].x * f, sum[i].y * f, sum[i].z * f,
                                                   sum[i].w * f));
                        }
                    }
                    if (join.all) break;
                    __syncwarp();
                    __stcg(a.part_ml + to, make_float2(m, l));
                    join = join_of_groups(p, width);
                }
                if (!ok) break;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&B.item_empty[it]);
        }
    }
    tc_before();
    __syncthreads();
    if (warp == 16) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                     : "memory");
    }
}

template <int D, bool BF>
sq_status launch_tiles(const PagedArgs &a, const void *k_cache, const void *v_cache, int sms,
                       cudaStream_t st) {
    using C = TilesCfg<D, BF>;
    static std::mutex mu;
    static bool done[64] = {};
    DeviceInfo di;
    sq_status rc = device_info(&di);
    if (rc != SQ_OK) return rc;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!done[di.device & 63]) {
            if (cudaFuncSetAttribute(paged_tiles_kernel<D, BF>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C::kSmem) != cudaSuccess)
                return SQ_ERR_CUDA;
            done[di.device & 63] = true;
        }
    }
    return launch_pdl(paged_tiles_kernel<D, BF>, dim3((unsigned)sms), dim3(kThreads), C::kSmem, st,
                      1, a, static_cast<const uint16_t *>(k_cache),
                      static_cast<const uint16_t *>(v_cache));
}

}  // namespace

sq_status launch_paged_tiles(const PagedArgs &a, const void *k_cache, const void *v_cache, int D,
                             bool bf16, int sms, cudaStream_t st) {
    if (D == 128)
        return bf16 ? launch_tiles<128, true>(a, k_cache, v_cache, sms, st)
                    : launch_tiles<128, false>(a, k_cache, v_cache, sms, st);
    return bf16 ? launch_tiles<64, true>(a, k_cache, v_cache, sms, st)
                : launch_tiles<64, false>(a, k_cache, v_cache, sms, st);
}

}  // namespace sq
