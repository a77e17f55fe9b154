// Host-only checks of the gated linear's grouped pair items (schedule.cuh), run on the
// CPU by tests/test_gated_schedule.py: every pair tile's columns are one item's whatever
// the group of row blocks is, and a group of one is the other linears' order; and that
// launches of few rows cover every column once.  Prints a summary; exit status 1 on a
// failure.
#include "schedule.cuh"

#include <cstdio>
#include <vector>

using namespace sq::sched;

static long long g_checked = 0, g_fail = 0;
static void check(bool ok, const char *what, long long a, long long b, long long c, long long d) {
    if (ok) return;
    if (g_fail++ < 20) std::printf("FAIL %s: %lld %lld %lld %lld\n", what, a, b, c, d);
}

static void pairs(int m_pairs, int n_tiles, int clusters, int group) {
    const PairSchedule sc = make_pair_schedule(m_pairs, n_tiles, clusters);
    std::vector<unsigned char> cover((size_t)m_pairs * n_tiles * 2, 0);
    for (int i = 0; i < sc.items; ++i) {
        int m0, n0, bn;
        grouped_item_at(sc, group, i, m0, n0, bn);
        const int m = m0 / (2 * BM);
        const bool in = m0 % (2 * BM) == 0 && n0 % 128 == 0 && m < m_pairs && n0 / BN < n_tiles &&
                        (bn == BN || bn == BN / 2);
        check(in, "item", m_pairs, n_tiles, clusters, i);
        for (int h = 0; in && h < bn / 128; ++h) ++cover[(size_t)m * n_tiles * 2 + n0 / 128 + h];
        if (group == 1) {
            int a, b, c;
            pair_item_at(sc, i, a, b, c);
            check(a == m0 && b == n0 && c == bn, "group of one", m_pairs, n_tiles, clusters, i);
        }
    }
    for (unsigned char n : cover) check(n == 1, "pair coverage", m_pairs, n_tiles, clusters, group);
    ++g_checked;
}

// Launches of few rows: every K block of every column is one unit's, columns in multiples
// of the gate's and the other projection's blocks together.
static void few_rows(long long M, long long N, long long K, int sms, bool split) {
    int grid = 0, tile_n = 0;
    const Schedule sc = plan_gated(M, N, K, sms, split, &grid, &tile_n);
    check(grid >= 1 && grid <= sms && tile_n % 64 == 0 && tile_n <= BN, "grid", M, N, K, sms);
    const int m_tiles = (int)((M + BM - 1) / BM);
    const int blocks = (int)((N + 63) / 64);
    std::vector<unsigned char> cover((size_t)m_tiles * blocks * sc.nkb, 0);
    for (int c = 0; c < grid; ++c) {
        Cursor cu;
        cursor_init(sc, cu, c);
        Work w;
        while (next_work(sc, cu, w, grid, tile_n)) {
            const bool in = w.m0 % BM == 0 && w.m0 / BM < m_tiles && w.n0 % 64 == 0 && w.n0 < N + BN &&
                            w.bn % 64 == 0 && w.bn <= BN && 0 <= w.kb0 && w.kb0 < w.kb1 &&
                            w.kb1 <= sc.nkb;
            check(in, "unit", M, N, K, c);
            for (int b = w.n0 / 64; in && b < blocks && b < (w.n0 + w.bn) / 64; ++b)
                for (int kb = w.kb0; kb < w.kb1; ++kb)
                    ++cover[((size_t)(w.m0 / BM) * blocks + b) * sc.nkb + kb];
        }
    }
    for (unsigned char n : cover) check(n == 1, "coverage", M, N, K, sms);
    ++g_checked;
}

int main() {
    for (long long M : {1, 16, 128, 129, 255, 256, 300})
        for (long long F : {1, 33, 64, 65, 1000, 4096, 5000, 9728, 9729, 11008, 12288, 14336, 14600})
            for (long long K : {64, 2048, 4096, 8192})
                for (int sms : {1, 2, 148, 152})
                    for (int split : {0, 1}) few_rows(M, (F + 31) / 32 * 64, K, sms, split != 0);

    for (int m : {1, 2, 7, 8, 9, 32, 33})
        for (int n : {1, 5, 40, 96, 97})
            for (int c : {1, 7, 76})
                for (int g : {1, 4, 8, 16}) pairs(m, n, c, g);
    std::printf("checked %lld launches, %lld failures\n", g_checked, g_fail);
    return g_fail ? 1 : 0;
}
