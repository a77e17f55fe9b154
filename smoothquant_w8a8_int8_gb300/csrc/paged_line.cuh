// The line of work of the attention kernels over the paged cache, and its
// division over the CTAs.  Host and device, so that it can be checked without
// a GPU.
//
// An item is a tile of query rows (tokens x heads of one key/value
// head's group) of one sequence and one key/value head; its keys are cut into
// tiles of KT.  All (item, key tile) pairs stand in one line -- sequences,
// then row tiles, then key/value heads, then key tiles -- each item's followed
// by PAD pairs without work that stand for the time of its start and end (none
// where all items are of one length, over a shared prefix), and worker c of n (a
// CTA, or a warp) takes pairs [c W / n, (c + 1) W / n): every worker has the same
// share whatever the lengths, known only on the device, are.  An item that lies in
// several workers' shares leaves one partial result (row maximum, sum,
// unnormalised output) per worker in the workspace; the one that arrives last
// (a counter) joins them in the order of the line, so that the result does not
// depend on who is last.  The line is shorter than 2^31 pairs (checked on the
// host for the longest that the sizes allow), but for sequences that overlap: see
// in_order.
#pragma once
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

namespace sq {

constexpr int kMaxWorkers = 2048;

struct PagedArgs {
    const float *Q;      // [T] rows of ldq floats, head h at column h D
    float *O;            // [T][Hq D]
    int64_t ldq;
    const int *block_table, *q_start, *kv_len, *prefix_pages;
    int64_t max_pages;
    float *prefix_o;     // [T Hq][D] unnormalised output over the prefix
    float2 *prefix_ml;   // [T Hq] its row maximum (log2 units) and sum
    unsigned *counters;  // zero between launches: kMaxWorkers of items, and as many of
                         // groups of an item's pieces
    float *part_o;       // [2 workers][rows][D] partial outputs, two slots each
    float2 *part_ml;     // [2 workers][rows]
    unsigned *error;     // the library's error word
    int T, B, Hq, Hkv, G;
    int tpt;             // tokens per row tile
    int g_inv;           // ceil(2^16 / G): n / G = n g_inv >> 16 for n < 256
    int num_pages, page_shift;
    int prefix_len;
    int kstart;          // first key of the suffix's first key tile
    int front_tiles;     // key tiles of the prefix in front of each item's own keys: 0
                         // where the prefix is a launch of its own
    int front_shift;     // front_tiles KT - kstart: 0, or KT for a prefix that ends in a tile
    int cap;             // keys a row of the page table can name
    float scale;         // a power of two; times q_factor the call's scale times log2 e
    float q_factor;      // what the queries are multiplied by, 0 for a scale of zero
    int prefix_phase;    // 1: every token over the prefix, into prefix_o / prefix_ml
    const float *k_scale, *v_scale;  // an int8 cache's: [cache rows]
    int after_prefix;    // 1: the few rows' launch behind that one (see begin_rows)
};

namespace {

#define SQ_HD __host__ __device__ __forceinline__

SQ_HD int load_int(const int *p) {
#ifdef __CUDA_ARCH__
    return __ldg(p);
#else
    return *p;
#endif
}
SQ_HD int at_most(int a, int b) { return a < b ? a : b; }
SQ_HD int at_least(int a, int b) { return a > b ? a : b; }

struct Seq {
    int q0, qlen, kv;  // first token, tokens, keys after the append
};
// The device arrays are taken as they come: offsets clamped into [0, T], a
// sequence's end to its start at least, lengths into [0, cap].
SQ_HD Seq load_seq(const PagedArgs &a, int b) {
    Seq s;
    const int e = a.prefix_phase ? a.B : b + 1;
    s.q0 = at_most(at_least(load_int(a.q_start + (a.prefix_phase ? 0 : b)), 0), a.T);
    s.qlen = at_most(at_least(load_int(a.q_start + e), s.q0), a.T) - s.q0;
    s.kv = a.prefix_phase ? a.prefix_len : at_most(at_least(load_int(a.kv_len + b), 0), a.cap);
    return s;
}
SQ_HD int row_tiles(const PagedArgs &a, const Seq &s) {
    return (s.qlen + a.tpt - 1) / a.tpt;
}
// One past the last key that any row of row tile j attends to (suffix: causal;
// a tile none of whose rows has a key gets one at or below zero).
SQ_HD int tile_keys(const PagedArgs &a, const Seq &s, int j) {
    return a.prefix_phase ? s.kv : s.kv - s.qlen + at_most(s.qlen, (j + 1) * a.tpt);
}
template <int KT>
SQ_HD int key_tiles(const PagedArgs &a, const Seq &s, int j) {
    const int n = tile_keys(a, s, j) - a.kstart;
    // at least one: its rows are written
    return a.front_tiles + (n <= KT ? 1 : (n + KT - 1) / KT);
}
// sum of floor((p i + q) / m) over i < n; m > 0, and m n + p + q < 2^32 (T and a
// row of the page table are limited to that).  The sum counts lattice points
// below a line: whole parts of p / m and q / m are summed in closed form, and
// what is left is the same sum with the axes exchanged.
SQ_HD int floor_sum(uint32_t n, uint32_t m, uint32_t p, uint32_t q) {
    uint32_t total = 0;  // the line is shorter than 2^31
#pragma unroll 1
    while (n > 0) {
        const uint32_t pm = p / m, qm = q / m;
        total += (uint32_t)((uint64_t)(n - 1) * n / 2) * pm + n * qm;
        p -= pm * m;
        q -= qm * m;
        const uint32_t top = p * n + q;
        if (top < m) break;
        n = top / m;
        q = top - n * m;
        const uint32_t was = m;
        m = p;
        p = was;
    }
    return (int)total;
}
// pairs of one key/value head's items over the first J row tiles
template <int KT, int PAD>
SQ_HD int pairs_before(const PagedArgs &a, const Seq &s, int J) {
    if (a.prefix_phase) return J * key_tiles<KT>(a, s, 0);
    const int tiles = row_tiles(a, s);
    const int whole = at_most(J, tiles - 1);  // the last row tile may hold fewer tokens
    int sum = J * PAD;
    if (whole > 0) {
        sum += whole * a.front_tiles;
        const int base = s.kv - s.qlen - a.kstart;
        // row tiles whose keys fit one key tile: base + (j + 1) tpt <= KT
        const int ones = at_most(KT < base ? 0 : (int)((uint32_t)(KT - base) / a.tpt), whole);
        sum += ones + floor_sum(whole - ones, KT, a.tpt, base + (ones + 1) * a.tpt + KT - 1);
    }
    if (J > whole && J > 0) sum += key_tiles<KT>(a, s, J - 1);
    return sum;
}

// Whether sequence b ends where it starts or behind it.  Where all do, they hold at
// most T tokens in all, and the host has checked the longest line of those.  Where one
// does not, sequences overlap, B of them with T tokens each at most: one sequence's
// pairs still fit, but their sum may wrap around, and nothing is worked on (see
// find_shares).
SQ_HD bool in_order(const PagedArgs &a, int b) {
    return a.prefix_phase || load_int(a.q_start + b) <= load_int(a.q_start + b + 1);
}

// Where a worker's share starts.
struct Share {
    int total;           // W
    int begin, end;      // this worker's pairs
    int seq, seq_begin;  // the sequence they begin in, and its position on the line
    int each, rest;      // W / n, rounded down, and what that leaves
    float per_pair;      // n / W
    int workers;         // workers that take a share
    int self;            // this worker
};
// The first pair of worker c: floor(c W / n)  (n < 2^16)
SQ_HD int share_begin(const Share &s, int c) {
    return s.each * c + (int)((uint32_t)s.rest * (uint32_t)c / (uint32_t)s.workers);
}
// the worker whose share holds position x: a guess that is off by one at most
// (three roundings of 2^-24, under 2^16 workers), put right
SQ_HD int share_of(const Share &s, int x) {
    int c = at_most((int)((float)x * s.per_pair), s.workers - 1);
    if (share_begin(s, c) > x) --c;
    else if (share_begin(s, c + 1) <= x) ++c;
    return c;
}
SQ_HD void set_shares(Share &s, int total, int workers, int self) {
    s.total = total;
    s.workers = workers;
    s.self = self;
    s.each = s.rest = 0;
    s.per_pair = 0.0f;
    s.begin = s.end = total;
    if (workers == 0) return;
    s.each = total / workers;
    s.rest = total - s.each * workers;
    s.per_pair = (float)workers / (float)total;
    if (self < workers) {
        s.begin = share_begin(s, self);
        s.end = share_begin(s, self + 1);
    }
}

// A worker's piece of an item.
struct Piece {
    int tok0, ntok;     // tokens of the row tile
    int head;           // key/value head
    int pos0;           // position of token tok0 (suffix)
    int key0, ntiles;   // first key and key tiles of the piece (see key_range)
    int keys;           // one past the last key any row attends to
    int seq;
    int first, npieces;  // first worker of the item; npieces = 1: the whole item
    int slot;           // the worker's partial slot
};

// An item's key tiles are numbered on: those of the prefix in front of the item's
// own, whose numbers end at kstart, and then its own from there.  The tile in
// which a prefix ends comes twice, once for the prefix and once for the
// sequence's own keys.
struct KeyRange {
    int key;      // the first key of the tile
    int lo, hi;   // keys of it that a row with `limit` keys sees: from lo, before hi
    bool front;   // the prefix's pages
};
SQ_HD KeyRange key_range(const PagedArgs &a, int key0, int limit) {
    KeyRange r;
    r.front = key0 < a.kstart;
    r.key = r.front ? key0 + a.front_shift : key0;
    r.lo = r.front || a.prefix_phase ? 0 : a.prefix_len;
    r.hi = r.front ? at_most(limit, a.prefix_len) : limit;
    r.front = r.front || a.prefix_phase;
    return r;
}

// A split item's pieces are joined by groups of neighbours and then the groups'
// sums, where one after the other would take longer than the second step (`most`:
// the pieces up to which it does not): 1216 warps' pieces of one head's 100,000
// keys took 240 us to join in one go.
struct Join {
    int first, step, n;  // pieces first, first + step, ...
    int counter;         // counts the arrivals of the n
    bool all;            // they are the whole item
};
SQ_HD int join_width(int npieces, int most) {
    return npieces <= most ? npieces : (int)ceilf(sqrtf((float)npieces));
}
// The join that piece c takes part in.  A group's counter is that of its last
// worker, which no other group ends in: the next item's first group, if it begins
// there, is longer.
SQ_HD Join join_of(const Piece &p, int c, int width) {
    Join j;
    j.all = width == p.npieces;
    j.first = c / width * width;
    j.step = 1;
    j.n = at_most(width, p.npieces - j.first);
    j.counter = j.all ? p.first : kMaxWorkers + p.first + j.first + j.n - 1;
    return j;
}
// The join of the groups' sums, which stand in the places of their first pieces.
SQ_HD Join join_of_groups(const Piece &p, int width) {
    Join j;
    j.all = true;
    j.first = 0;
    j.step = width;
    j.n = (p.npieces + width - 1) / width;
    j.counter = p.first;
    return j;
}

// Walks the pieces of a worker's share.
template <int KT, int PAD>
struct Walk {
    int at, end;  // position, end of the share
    int b, j, h, k;
    int tiles, nk, pad;
    Seq s;

    SQ_HD void start(const PagedArgs &a, const Share &sh) {
        pad = a.prefix_phase ? 0 : PAD;
        at = sh.begin;
        end = sh.end;
        if (at >= end) return;
        b = sh.seq;
        s = load_seq(a, b);
        tiles = row_tiles(a, s);
        const int rem = at - sh.seq_begin;
        int hi = tiles - 1, before = 0;
        j = 0;  // the last row tile that starts at or before rem
#pragma unroll 1
        while (j < hi) {
            const int mid = (j + hi + 1) / 2;
            const int n = a.Hkv * pairs_before<KT, PAD>(a, s, mid);
            if (n <= rem) {
                j = mid;
                before = n;
            } else {
                hi = mid - 1;
            }
        }
        nk = key_tiles<KT>(a, s, j);
        const int r = rem - before;  // Hkv items of one length
        h = (int)((uint32_t)r / (uint32_t)(nk + pad));
        k = r - h * (nk + pad);
    }
    // the next piece, or false at the end of the share
    SQ_HD bool next(const PagedArgs &a, const Share &sh, Piece &p) {
        if (at < end && k >= nk) {
            // past an item's work: over its pairs without work to the next item
            at += nk + pad - k;
            k = 0;
            if (++h == a.Hkv) {
                h = 0;
                ++j;
#pragma unroll 1
                while (j >= tiles && b < a.B - 1 && at < end) {  // the next sequence with a row
                    s = load_seq(a, ++b);
                    tiles = row_tiles(a, s);
                    j = 0;
                }
                if (j < tiles) nk = key_tiles<KT>(a, s, j);
            }
        }
        if (at >= end) return false;
        const int take = at_most(end - at, nk - k);
        const int s0 = at - k;
        p.tok0 = s.q0 + j * a.tpt;
        p.ntok = at_most(a.tpt, s.qlen - j * a.tpt);
        p.head = h;
        p.pos0 = s.kv - s.qlen + j * a.tpt;
        p.key0 = a.kstart + (k - a.front_tiles) * KT;
        p.ntiles = take;
        p.keys = tile_keys(a, s, j);
        p.seq = b;
        // the item's other ends, where they are not this worker's
        p.first = k == 0 ? sh.self : share_of(sh, s0);
        const int last = k + take == nk ? sh.self : share_of(sh, s0 + nk - 1);
        p.npieces = last - p.first + 1;
        p.slot = k == 0 ? 1 : 0;  // begun here: slot 1; begun before: slot 0
        at += take;
        k += take;
        return true;
    }
};

}  // namespace
}  // namespace sq
