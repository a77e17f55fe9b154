// Host-only check of the paged attention's division of work (paged_line.cuh),
// run on the CPU by tests/test_paged_line.py: for random batches, head counts,
// tile sizes and worker counts, the pieces that all workers walk cover every (row
// tile, key/value head, key tile) exactly once, in order; the pieces of a split
// item name the workers that hold them, two partial slots per worker are enough, and
// the counter of a split item is nobody else's.  Prints a summary line; exit
// status 1 on any failure.
#include "paged_line.cuh"

#include <cstdio>
#include <map>
#include <random>
#include <tuple>
#include <vector>

using namespace sq;

static long long g_checked = 0, g_fail = 0;
#define CHECK(cond)                                              \
    do {                                                         \
        ++g_checked;                                             \
        if (!(cond) && g_fail++ < 20)                            \
            std::printf("FAIL line %d: %s\n", __LINE__, #cond);  \
    } while (0)

template <int KT, int PAD>
static void check(PagedArgs a, int grid, int min_pairs, int most) {
    // the line, pair by pair, as the header's comment states it
    const int nb = a.prefix_phase ? 1 : a.B;
    std::vector<std::tuple<int, int, int, int>> line;  // (sequence, row tile, head, key tile)
    std::vector<int64_t> seq_begin;
    for (int b = 0; b < nb; ++b) {
        const Seq s = load_seq(a, b);
        CHECK(s.q0 >= 0 && s.qlen >= 0 && s.q0 + s.qlen <= a.T && s.kv >= 0);
        seq_begin.push_back((int64_t)line.size());
        for (int j = 0; j < row_tiles(a, s); ++j) {
            int last = 0;  // keys of the tile's last token, one past
            for (int i = j * a.tpt; i < std::min(s.qlen, (j + 1) * a.tpt); ++i)
                last = a.prefix_phase ? a.prefix_len : s.kv - s.qlen + i + 1;
            int n = 1;
            while (a.kstart + n * KT < last) ++n;
            n += a.front_tiles;
            CHECK(n == key_tiles<KT>(a, s, j));
            // its tiles hold every key that it attends to (here) once, in order
            int key = a.prefix_phase || a.front_tiles ? 0 : a.prefix_len;
            for (int k = 0; k < n; ++k) {
                const KeyRange r = key_range(a, a.kstart + (k - a.front_tiles) * KT, last);
                const int lo = std::max(r.lo, r.key), hi = std::min(r.hi, r.key + KT);
                CHECK(r.key >= 0 && r.key % KT == 0);
                CHECK(r.front == (a.prefix_phase || lo < a.prefix_len));
                if (lo >= hi) continue;
                CHECK(lo == key);
                key = hi;
            }
            CHECK(last <= key);
            for (int h = 0; h < a.Hkv; ++h)
                for (int k = 0; k < n + (a.prefix_phase ? 0 : PAD); ++k)  // the last without work
                    line.emplace_back(b, j, h, k < n ? k : -1);
        }
        const int64_t pairs = pairs_before<KT, PAD>(a, s, row_tiles(a, s));
        CHECK(a.Hkv * pairs == (int64_t)line.size() - seq_begin[b]);
    }
    const int64_t total = (int64_t)line.size();
    if (total == 0) return;
    const int64_t fit = (total + min_pairs - 1) / min_pairs;
    const int workers = fit < grid ? (int)fit : grid;
    int64_t at = 0;
    std::map<int, std::tuple<int, int, int>> counter;          // first worker -> split item
    std::map<std::tuple<int, int, int>, std::vector<int>> parts;  // split item -> workers
    std::map<std::tuple<int, int, int>, int> want;
    for (int c = 0; c < workers; ++c) {
        Share sh;
        set_shares(sh, (int)total, workers, c);
        CHECK(sh.begin == total * c / workers && sh.end == total * (c + 1) / workers);
        CHECK(sh.begin == at && sh.end > sh.begin);
        sh.seq = 0;
        for (int b = 0; b < nb; ++b)
            if (seq_begin[b] <= sh.begin &&
                (b + 1 == nb ? total : seq_begin[b + 1]) > seq_begin[b])
                sh.seq = b;
        sh.seq_begin = (int)seq_begin[sh.seq];
        Walk<KT, PAD> w;
        w.start(a, sh);
        Piece p;
        bool slots[2] = {false, false};
        auto idle = [&]() {  // pairs without work that stand next in the share
            while (at < sh.end && std::get<3>(line[at]) < 0) ++at;
        };
        for (idle(); w.next(a, sh, p); idle()) {
            const auto [b, j, h, k] = line[at];
            const Seq s = load_seq(a, b);
            CHECK(p.seq == b && p.head == h && p.ntiles >= 1);
            CHECK(p.tok0 == s.q0 + j * a.tpt && p.ntok == std::min(a.tpt, s.qlen - j * a.tpt));
            CHECK(p.key0 == a.kstart + (k - a.front_tiles) * KT);
            CHECK(p.keys == tile_keys(a, s, j));
            if (!a.prefix_phase) CHECK(p.pos0 == s.kv - s.qlen + j * a.tpt);
            for (int i = 0; i < p.ntiles; ++i)
                CHECK(at + i < total && line[at + i] == std::make_tuple(b, j, h, k + i));
            const auto item = std::make_tuple(b, j, h);
            const bool whole = k == 0 && p.ntiles == key_tiles<KT>(a, s, j);
            CHECK(whole == (p.npieces == 1));
            if (!whole) {
                CHECK(p.slot >= 0 && p.slot < 2 && !slots[p.slot]);
                slots[p.slot] = true;
                // the joiner reads slot 1 of the first worker and slot 0 of the others
                CHECK((c == p.first) == (p.slot == 1));
                CHECK(!counter.count(p.first) || counter[p.first] == item);
                counter[p.first] = item;
                parts[item].push_back(c);
                want[item] = p.npieces;
                CHECK(parts[item].size() ==
                      (size_t)(c - p.first + 1));  // every worker between holds a piece
            }
            at += p.ntiles;
        }
        CHECK(at == sh.end);
    }
    CHECK(at == total);
    for (auto &e : parts) CHECK((int)e.second.size() == want[e.first]);
    // the joins: every piece once, in groups whose counters are nobody else's
    std::map<int, std::tuple<std::tuple<int, int, int>, int>> group;
    for (auto &e : parts) {
        Piece p;
        p.first = e.second[0];
        p.npieces = (int)e.second.size();
        const int width = join_width(p.npieces, most);
        CHECK(width >= 1 && (width == p.npieces) == (p.npieces <= most));
        int pieces = 0;
        for (int c = 0; c < p.npieces; ++c) {
            const Join j = join_of(p, c, width);
            CHECK(j.first <= c && c < j.first + j.n && j.step == 1 && j.n <= width);
            CHECK(j.first + j.n <= p.npieces && j.all == (p.npieces <= most));
            CHECK(j.counter >= 0 && j.counter < 2 * kMaxWorkers);
            const auto who = std::make_tuple(e.first, j.first);
            CHECK(!group.count(j.counter) || group[j.counter] == who);
            group[j.counter] = who;
            if (c == j.first) pieces += j.n;
            if (j.all) continue;
            const Join k = join_of_groups(p, width);
            CHECK(j.first % k.step == 0 && j.first / k.step < k.n && k.all && k.first == 0);
            CHECK((k.n - 1) * k.step < p.npieces && k.n * k.step >= p.npieces);
            CHECK(k.counter == p.first);
        }
        CHECK(pieces == p.npieces);
    }
    Share sh;
    set_shares(sh, (int)total, workers, 0);
    for (int64_t x = 0; x < total; x += 1 + total / 97) {
        const int c = share_of(sh, (int)x);
        CHECK(c >= 0 && c < workers && total * c / workers <= x &&
              x < total * (c + 1) / workers);
    }
}

int main() {
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int trial = 0; trial < 4000; ++trial) {
        PagedArgs a = {};
        a.B = pick(1, trial % 3 ? 6 : 40);
        a.Hkv = pick(1, 4);
        a.G = pick(1, 8);
        const int rows = trial % 2 ? 256 : (trial % 4 ? 8 : 16);
        a.tpt = std::max(1, rows / a.G);
        const int KT = trial % 2 ? 128 : 16;
        const int page = 16 << pick(0, 4);
        a.max_pages = pick(0, 3000 / page);
        a.cap = (int)(a.max_pages * page);
        std::vector<int> q(a.B + 1), kv(a.B);
        q[0] = pick(0, 3);
        const int longest = pick(0, 2) ? pick(0, 5) : pick(0, 700);
        for (int b = 0; b < a.B; ++b) {
            q[b + 1] = q[b] + pick(0, longest);
            kv[b] = pick(0, 4) ? pick(0, 2500) : 0;
        }
        a.T = q[a.B] + pick(0, 5);
        if (trial % 11 == 0)  // arrays that hold anything
            for (int b = 0; b < a.B; ++b) {
                q[pick(0, a.B)] = (int)rng();
                kv[b] = (int)rng();
            }
        a.q_start = q.data();
        a.kv_len = kv.data();
        a.prefix_len = pick(0, 1) ? pick(1, 1500) : 0;
        for (int phase = a.prefix_len ? 1 : 0; phase >= 0; --phase) {
            a.prefix_phase = phase;
            a.kstart = phase ? 0 : a.prefix_len / KT * KT;
            // the prefix in front of every item's own keys, or not
            a.front_tiles = phase || trial % 5 < 2 ? 0 : (a.prefix_len + KT - 1) / KT;
            a.front_shift = a.front_tiles ? a.front_tiles * KT - a.kstart : 0;
            const int grid = pick(1, 152), least = pick(1, 4), most = pick(2, 16);
            if (KT == 16) check<16, 2>(a, grid, least, most);
            else trial % 4 == 1 ? check<128, 4>(a, grid, least, most)
                                : check<128, 6>(a, grid, least, most);
        }
    }
    // the closed-form sum against a loop
    for (int trial = 0; trial < 20000; ++trial) {
        const int n = pick(0, 60), m = pick(1, 130), p = pick(0, 300), q = pick(0, 3000);
        int64_t want = 0;
        for (int i = 0; i < n; ++i) want += (p * i + q) / m;
        CHECK(floor_sum(n, m, p, q) == want);
    }
    std::printf("%lld checks, %lld failures\n", g_checked, g_fail);
    return g_fail != 0;
}
