// Goes through csrc/mx_plan.h as the pairs of CTAs do, for lists of problems of all kinds: every
// stage of every tile is taken once, and the pieces of a tile find each other.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "mx_plan.h"

using namespace kfac::mx;

namespace {

struct Params : Deal {
    Tiles prob[MAX_PROBS];
};

int failed = 0;
void need(bool ok, const char *what, long long a = 0, long long b = 0) {
    if (!ok && ++failed < 20) std::printf("%s (%lld, %lld)\n", what, a, b);
}

double slack = 0;

void go(std::vector<Tiles> list, int most) {
    std::stable_sort(list.begin(), list.end(), [](const Tiles &a, const Tiles &b) { return a.k_tiles > b.k_tiles; });
    for (int at = 0; at < (int)list.size();) {
        const Launch l = make_launch(list, at, most);
        need(l.to > at && l.pairs >= 1 && l.pairs <= most, "launch", l.to, l.pairs);
        if (l.to <= at) return;
        Params P;
        static_cast<Deal &>(P) = l.deal;
        for (int i = 0; i < P.nprob; ++i) P.prob[i] = l.tiles[i];
        std::map<std::tuple<int, int, int>, std::vector<std::pair<int, int>>> taken;
        std::map<int, std::set<int>> slots;                    // pieces of the tile that begins there, by slot
        std::map<int, Pieces> pieces;
        std::set<int> used;
        long long most_stages = 0, all_stages = 0;
        for (int pair = 0; pair < l.pairs; ++pair) {
            Walk walk(P, pair, l.pairs);
            long long mine = 0;
            for (Item k; walk.next(P, k);) {
                const Tiles &q = P.prob[k.p];
                need(k.tm >= 0 && k.tm < q.tiles_m && k.tn >= 0 && k.tn < q.tiles_n && (!q.sym || k.tn >= k.tm), "tile", k.tm, k.tn);
                need(0 <= k.kt0 && (k.kt0 < k.kt1 || q.k_tiles == 0) && k.kt1 <= q.k_tiles, "stages", k.kt0, k.kt1);
                need(!k.piece || k.kt1 - k.kt0 >= MIN_PIECE / 2, "piece", k.kt0, k.kt1);
                taken[{k.p, k.tm, k.tn}].push_back({k.kt0, k.kt1});
                mine += k.kt1 - k.kt0;
                if (k.piece) {
                    const Pieces r = pieces_of(P, k.begin, q.k_tiles, pair);
                    const int slot = 2 * pair + (k.kt0 == 0);
                    need(used.insert(slot).second, "slot used twice", slot);
                    need((k.kt0 == 0) == (pair == r.first), "the first piece", pair, r.first);
                    slots[k.begin].insert(slot);
                    if (pieces.count(k.begin)) {
                        const Pieces &o = pieces[k.begin];
                        need(o.first == r.first && o.last == r.last && o.count == r.count, "pieces agree", r.first, r.last);
                    }
                    pieces[k.begin] = r;
                }
            }
            most_stages = std::max(most_stages, mine);
            all_stages += mine;
        }
        std::set<int> firsts;
        for (auto &t : pieces) {
            need((int)slots[t.first].size() == t.second.count, "number of pieces", t.second.count, slots[t.first].size());
            need(firsts.insert(t.second.first).second, "counter used twice", t.second.first);
        }
        for (int i = 0; i < P.nprob; ++i) {
            const Tiles &q = P.prob[i];
            for (int tm = 0; tm < q.tiles_m; ++tm)
                for (int tn = q.sym ? tm : 0; tn < q.tiles_n; ++tn) {
                    auto &v = taken[{i, tm, tn}];
                    std::sort(v.begin(), v.end());
                    int to = 0;
                    for (auto &x : v) {
                        need(x.first == to, "a stage twice or never", x.first, to);
                        to = x.second;
                    }
                    need(to == q.k_tiles && (q.k_tiles > 0 || v.size() == 1), "all stages", to, q.k_tiles);
                    taken.erase({i, tm, tn});
                }
        }
        need(taken.empty(), "no other tile");
        if (l.span) slack = std::max(slack, (double)most_stages - (double)all_stages / l.pairs);
        at = l.to;
    }
}

}  // namespace

int main() {
    std::mt19937 rng(7);
    auto pick = [&](int a, int b) { return a + (int)(rng() % (unsigned)(b - a + 1)); };
    for (int tm = 1; tm < 20; ++tm)
        for (int k : {0, 1, 9, 23, 24, 40, 64, 128, 700})
            for (int sym : {0, 1}) go({Tiles{tm, sym ? tm : pick(1, 20), k, sym, 0, 0}}, 76);
    for (int n = 0; n < 4000; ++n) {
        std::vector<Tiles> list;
        for (int i = pick(1, n % 10 ? 8 : 120); i > 0; --i) {
            const int tm = pick(1, 12), sym = pick(0, 1);
            list.push_back(Tiles{tm, sym ? tm : pick(1, 12), pick(0, 3) ? pick(0, 30) : pick(0, 300), sym, 0, 0});
        }
        go(list, n % 3 ? 76 : pick(1, MAX_PAIRS));
    }
    std::printf("largest slack %g stages, %d failed\n", slack, failed);
    return failed != 0;
}
