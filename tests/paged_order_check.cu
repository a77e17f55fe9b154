// Host-only check of the paged attention's line of work (paged_line.cuh) over what
// paged_line_check.cu leaves out, run on the CPU by tests/test_paged_order.py:
//  - row tiles of 128, 16 and 8 rows with every number of heads to a group up to
//    them, as the launches have them;
//  - any q_start: where every sequence is in order, the pairs of all stay within what
//    the host's check of the sizes has counted.  Where one is not, they overlap and can
//    pass 2^31 although that check holds: the shares are cut from a length of 0 then,
//    and no worker takes a piece.
#define main line_main
#include "paged_line_check.cu"
#undef main

#include <algorithm>

template <int KT, int PAD>
static bool any_order(const PagedArgs &a) {
    // the host's check, as launch_paged_attention makes it
    const int64_t tiles = (a.T + a.tpt - 1) / a.tpt + a.B;
    const int64_t keys = (a.cap + (int64_t)a.prefix_len) / KT + 16;
    if (tiles * a.Hkv > ((int64_t)1 << 31) / keys) return false;
    int64_t total = 0;
    bool ordered = true;
    for (int b = 0; b < a.B; ++b) {
        const Seq s = load_seq(a, b);
        CHECK(s.q0 >= 0 && s.qlen >= 0 && s.q0 + s.qlen <= a.T && s.kv >= 0 && s.kv <= a.cap);
        const int64_t n = (int64_t)a.Hkv * pairs_before<KT, PAD>(a, s, row_tiles(a, s));
        CHECK(n >= 0 && n < ((int64_t)1 << 31));  // one sequence's pairs fit
        total += n;
        ordered = ordered && in_order(a, b);
    }
    const bool fits = total < ((int64_t)1 << 31);
    CHECK(!ordered || (fits && total <= tiles * a.Hkv * keys));
    Share sh;
    sh.seq = sh.seq_begin = 0x55555555;  // never looked at
    set_shares(sh, 0, 0, a.B % 7);
    Walk<KT, PAD> w;
    w.start(a, sh);
    Piece p;
    CHECK(!w.next(a, sh, p));
    return !fits;
}

int main() {
    std::mt19937 rng(11);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int trial = 0; trial < 1500; ++trial) {
        const int kind = trial % 3, rows = kind == 0 ? 128 : kind == 1 ? 16 : 8;
        PagedArgs a = {};
        a.B = pick(1, 12);
        a.Hkv = pick(1, 3);
        a.G = pick(1, rows);
        a.tpt = rows / a.G;
        a.max_pages = pick(0, 40);
        a.cap = (int)a.max_pages * 64;
        std::vector<int> q(a.B + 1), kv(a.B);
        q[0] = pick(0, 3);
        const int longest = pick(0, 3) ? pick(0, 5) : pick(0, 400);
        for (int b = 0; b < a.B; ++b) {
            q[b + 1] = q[b] + pick(0, longest);
            kv[b] = pick(0, 4) ? pick(0, 2500) : 0;
        }
        a.T = q[a.B] + pick(0, 5);
        a.q_start = q.data();
        a.kv_len = kv.data();
        a.prefix_len = pick(0, 1) ? pick(1, 1500) : 0;
        const int KT = rows == 128 ? 128 : 16;
        for (int phase = a.prefix_len ? 1 : 0; phase >= 0; --phase) {
            a.prefix_phase = phase;
            a.kstart = phase ? 0 : a.prefix_len / KT * KT;
            a.front_tiles = phase || trial % 5 < 2 ? 0 : (a.prefix_len + KT - 1) / KT;
            a.front_shift = a.front_tiles ? a.front_tiles * KT - a.kstart : 0;
            const int grid = pick(1, 152), least = pick(1, 4), most = pick(2, 16);
            if (KT == 16) check<16, 2>(a, grid, least, most);
            else trial % 2 ? check<128, 4>(a, grid, least, most)
                           : check<128, 6>(a, grid, least, most);
        }
    }
    int too_long = 0;
    for (int trial = 0; trial < 600; ++trial) {
        const int rows = trial % 2 ? 128 : 8, KT = rows == 128 ? 128 : 16;
        PagedArgs a = {};
        a.B = 1 << pick(0, 11);
        a.T = 1 << pick(0, 13);
        a.Hkv = 1 << pick(0, 4);
        a.G = pick(1, rows);
        a.tpt = rows / a.G;
        a.max_pages = pick(1, 512);
        a.cap = (int)a.max_pages * 256;
        a.prefix_len = trial % 3 == 0 ? pick(1, 5000) : 0;
        std::vector<int> q(a.B + 1), kv(a.B);
        for (int b = 0; b <= a.B; ++b)
            q[b] = trial % 5 == 0 ? (int)rng() : b % 2 ? a.T : 0;  // 0, T, 0, T, ...
        if (trial % 3 == 1) std::sort(q.begin(), q.end());
        for (int b = 0; b < a.B; ++b) kv[b] = trial % 7 == 0 ? (int)rng() : a.cap;
        a.q_start = q.data();
        a.kv_len = kv.data();
        a.kstart = a.prefix_len / KT * KT;
        too_long += KT == 16 ? any_order<16, 2>(a) : any_order<128, 4>(a);
    }
    CHECK(too_long > 20);
    std::printf("%lld checks, %lld failures, %d lines too long\n", g_checked, g_fail, too_long);
    return g_fail != 0;
}
