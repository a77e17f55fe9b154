// Host-only checks of the gated linear's grouped pair items (schedule.cuh), run on the
// CPU by tests/test_gated_schedule.py: every pair tile's columns are one item's whatever
// the group of row blocks is, and a group of one is the other linears' order.  Prints a
// summary; exit status 1 on a failure.
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

int main() {
    for (int m : {1, 2, 7, 8, 9, 32, 33})
        for (int n : {1, 5, 40, 96, 97})
            for (int c : {1, 7, 76})
                for (int g : {1, 4, 8, 16}) pairs(m, n, c, g);
    std::printf("checked %lld launches, %lld failures\n", g_checked, g_fail);
    return g_fail ? 1 : 0;
}
