// mx_plan.h -- how the tiles of a launch of checkpoints' products are dealt out to pairs of
// CTAs, apart from the kernel, so that a host test can go through it.
#pragma once

#include <algorithm>
#include <vector>

#ifdef __CUDACC__
#define KFAC_PLAN_FN __host__ __device__ __forceinline__
#else
#define KFAC_PLAN_FN inline
#endif

namespace kfac {
namespace mx {

constexpr int MAX_PROBS = 46, MAX_PAIRS = 96, GROUP = 8;
// A tile is split only where that saves more than the pieces cost (their way through memory and the
// adding up by one CTA: 11 us = 40 stages), and not into pieces of under 12 stages.  16 tiles of 128
// stages: 57 us whole, 40 split; 64 tiles of 64 stages: 37 whole, 45 split.
constexpr int MIN_PIECE = 12, SPLIT_COST = 40;

KFAC_PLAN_FN int least(int a, int b) { return a < b ? a : b; }

// A problem's tiles.
struct Tiles {
    int tiles_m, tiles_n, k_tiles;  // k_tiles: stages of a tile
    int sym;                        // the upper ones only
    int first;                      // number of its first tile among all problems' tiles
    int span_begin;                 // where its tiles begin in the shared span
    int count() const { return sym ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n; }
};

// How the tiles are dealt out: tile by tile in turn up to `whole` (a multiple of the number of
// pairs, or all of the tiles that are worth splitting); then the tiles up to `short_first`, which
// would leave pairs idle in their last round, as one span of stages in equal shares (`share`: where
// each pair's ends), so that a tile may be in several pieces; then tiles of few stages in turn again.
struct Deal {
    int nprob, whole, short_first, total;
    int share[MAX_PAIRS];
};

struct Item {
    int p, tm, tn, kt0, kt1;
    bool piece;  // of a tile in several pieces
    int begin;   // of the tile in the span
};

// Tile number u of a problem: bands of GROUP rows of tiles, column by column, so that the CTAs
// at work together share panels of both operands in L2; of a symmetric result the upper tiles.
KFAC_PLAN_FN void place_tile(const Tiles &q, int u, Item &k) {
    const int T = q.tiles_n;
    if (q.sym) {
        int b0 = 0, gb;
        for (;;) {
            gb = least(GROUP, T - b0);
            const int size = gb * (T - b0) - gb * (gb - 1) / 2;
            if (u < size) break;
            u -= size;
            b0 += gb;
        }
        const int stair = gb * (gb + 1) / 2;
        if (u < stair) {
            int c = 0;
            while (u > c) u -= ++c;
            k.tn = b0 + c;
            k.tm = b0 + u;
        } else {
            u -= stair;
            k.tn = b0 + gb + u / gb;
            k.tm = b0 + u % gb;
        }
    } else {
        const int band = u / (GROUP * T), b0 = band * GROUP, gb = least(GROUP, q.tiles_m - b0);
        u -= b0 * T;
        k.tn = u / gb;
        k.tm = b0 + u % gb;
    }
}

// A pair's items, in turn.
struct Walk {
    int tile, step, at, end;
    template <class Params>
    KFAC_PLAN_FN Walk(const Params &P, int pair, int pairs)
        : tile(pair), step(pairs), at(pair ? P.share[pair - 1] : 0), end(P.share[pair]) {}
    template <class Params>
    KFAC_PLAN_FN bool next(const Params &P, Item &k) {
        const bool shared = tile >= P.whole && at < end;
        if (!shared && tile >= P.whole && tile < P.short_first)
            tile += (P.short_first - tile + step - 1) / step * step;  // (past what the shares hold)
        if (!shared && tile >= P.total) return false;
        int lo = 0, hi = P.nprob - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (shared ? P.prob[mid].span_begin <= at : P.prob[mid].first <= tile) lo = mid;
            else hi = mid - 1;
        }
        const Tiles &q = P.prob[lo];
        k.p = lo;
        k.piece = false;
        k.kt0 = 0;
        k.kt1 = q.k_tiles;
        if (shared) {
            const int n = (at - q.span_begin) / q.k_tiles;
            k.begin = q.span_begin + n * q.k_tiles;
            k.kt0 = at - k.begin;
            k.kt1 = least(q.k_tiles, end - k.begin);
            k.piece = k.kt1 - k.kt0 < q.k_tiles;
            at = k.begin + k.kt1;
            place_tile(q, n + (P.whole > q.first ? P.whole - q.first : 0), k);
        } else {
            place_tile(q, tile - q.first, k);
            tile += step;
        }
        return true;
    }
};

// The pairs whose shares have pieces of a tile of the span, and how many pieces there are (shares may be empty).
struct Pieces {
    int first, last, count;
};
KFAC_PLAN_FN Pieces pieces_of(const Deal &P, int begin, int stages, int pair) {
    Pieces r{pair, pair, 1};
    while (r.first > 0 && P.share[r.first - 1] > begin) {
        --r.first;
        r.count += P.share[r.first] > (r.first ? P.share[r.first - 1] : 0);
    }
    while (P.share[r.last] < begin + stages) {
        ++r.last;
        r.count += P.share[r.last] > P.share[r.last - 1];
    }
    return r;
}

// One launch: the problems from .. to - 1 of a list that has those of the most stages first.
struct Launch {
    int from, to, pairs, span;
    Deal deal;
    std::vector<Tiles> tiles;
};

inline Launch make_launch(const std::vector<Tiles> &list, int from, int most) {
    Launch l{};
    Deal &d = l.deal;
    l.from = l.to = from;
    long long total = 0;
    int longs = 0;  // tiles of enough stages to be split
    for (; l.to < (int)list.size() && l.to - from < MAX_PROBS; ++l.to) {
        Tiles t = list[l.to];
        if (total + t.count() > 0x3fffffffLL) break;
        t.first = (int)total;
        total += t.count();
        if (t.k_tiles >= 2 * MIN_PIECE) longs = (int)total;
        l.tiles.push_back(t);
    }
    d.nprob = l.to - from;
    d.total = (int)total;
    d.short_first = longs;
    d.whole = longs / most * most;
    l.pairs = std::max(1, std::min(d.total, most));
    // the stages of the tiles that are left, and what each pair has of the rounds before
    long long span = 0;
    std::vector<long long> mine(most, 0);
    int longest = 0;
    for (Tiles &t : l.tiles) {
        t.span_begin = (int)std::min<long long>(span, 0x7fffffff);
        const int end = t.first + t.count(), k = t.k_tiles;
        for (int p = 0; p < most && t.first < d.whole; ++p) {  // the tiles p, p + most, ...
            const int a = t.first + ((p - t.first) % most + most) % most, b = std::min(end, d.whole);
            if (a < b) mine[p] += (long long)((b - 1 - a) / most + 1) * k;
        }
        const int left = std::min(end, longs) - std::max(t.first, d.whole);
        if (left > 0) {
            span += (long long)left * k;
            longest = std::max(longest, k);
        }
    }
    const int left = longs - d.whole;
    if (left == 0 || span >= 0x7fffffff || (1.0 - (double)left / most) * longest <= SPLIT_COST) {
        d.whole = longs;
        return l;
    }
    l.span = (int)span;
    // as many pairs take part as have a piece's worth
    const int sharing = (int)std::min<long long>(most, std::max<long long>(1, span / MIN_PIECE));
    l.pairs = d.whole ? most : std::max(sharing, std::min(most, d.total - longs));
    double sum = (double)span, at = 0;
    for (int p = 0; p < sharing; ++p) sum += (double)mine[p];
    size_t i = 0;
    for (int p = 0; p < l.pairs; ++p) {
        const int before = p ? d.share[p - 1] : 0;
        if (p < sharing) at = std::min((double)span, at + std::max(0.0, sum / sharing - (double)mine[p]));
        int end = p + 1 >= sharing ? (int)span : (int)at;
        // a share ends at a tile's edge where it comes near one, and is empty where it would be very small
        while (i + 1 < l.tiles.size() && l.tiles[i + 1].span_begin <= end && l.tiles[i + 1].first < longs) ++i;
        const int k = l.tiles[i].k_tiles, in = (end - l.tiles[i].span_begin) % k;
        if (in < MIN_PIECE / 2) end -= in;
        else if (k - in < MIN_PIECE / 2) end += k - in;
        d.share[p] = end - before < MIN_PIECE / 2 && end < span ? before : end;
    }
    return l;
}

}  // namespace mx
}  // namespace kfac
