// Goes through the waits of csrc/ring.h with a model of a stage's barrier: every
// order in which the stage's events can fall between the waiting thread's steps.
#include <cstdio>
#include <vector>

#include "ring.h"

namespace {

// What happens to a stage, in order, from the row before row n on: given to it, its
// bytes land, it is consumed (the team that took it releases the stage), given to
// row n, row n's bytes land.
enum { GIVEN_BEFORE = 1, LANDED_BEFORE, CONSUMED, GIVEN, LANDED, EVENTS = LANDED };

struct Choices {  // the next path through a tree of choices
    std::vector<int> taken, of;
    size_t at = 0;
    int pick(int n) {
        if (at == taken.size()) {
            taken.push_back(0);
            of.push_back(n);
        }
        return taken[at++];
    }
    bool next() {
        while (!taken.empty() && taken.back() + 1 == of.back()) {
            taken.pop_back();
            of.pop_back();
        }
        if (taken.empty()) return false;
        ++taken.back();
        at = 0;
        return true;
    }
};

struct Stage {
    Choices &c;
    long long n;
    int stages, event, last;  // `last`: no event after this one ever comes
    void step() { event += c.pick(last - event + 1); }  // any number of events between two steps
    long long given() {
        step();
        return event >= GIVEN ? n : event >= GIVEN_BEFORE ? n - stages : -1;
    }
    // phases completed: n / stages of them before row n's own
    long long complete() const { return n / stages - (event < LANDED_BEFORE && n >= stages) + (event >= LANDED); }
    bool passes(int parity) const { return (complete() & 1) != parity; }
    bool wait_full(int parity) {
        step();
        while (!passes(parity) && event < last) ++event;
        return passes(parity);
    }
    void start() {}
    bool late() {  // (something happens before a spinning thread looks again, or nothing ever will)
        if (event == last) return true;
        ++event;
        return false;
    }
    // the warp's other threads: `others` says whether their waits ended
    bool others = true;
    int reads = 0;
    bool all(bool ok) const { return ok && others; }
    long long row() {
        ++reads;
        return event >= GIVEN ? n : -1000;  // (what stands there before is another row's, or nothing's)
    }
};

int failures = 0;
void check(bool ok, const char *what, long long n, int stages, int begin, int last) {
    if (ok) return;
    if (failures++ < 5) std::printf("%s: row %lld, %d stages, from event %d to %d\n", what, n, stages, begin, last);
}

}  // namespace

int main() {
    long long paths = 0;
    for (int stages = 2; stages <= 4; ++stages)
        for (long long n = 0; n < 4 * stages; ++n)
            for (int begin = n < stages ? CONSUMED : 0; begin <= EVENTS; ++begin)
                for (int last = begin; last <= EVENTS; ++last) {
                    Choices c;
                    do {
                        c.at = 0;
                        Stage s{c, n, stages, begin, last};
                        const bool held = kfac::loss::wait_stage(s, n, stages);
                        check(!held || s.event >= LANDED, "returned before the row had landed", n, stages, begin, last);
                        check(held || last < LANDED, "gave up although the row landed", n, stages, begin, last);
                        ++paths;
                    } while (c.next());
                    c = Choices{};
                    do {
                        c.at = 0;
                        Stage s{c, n, stages, begin, last};
                        s.others = c.pick(2) == 0;
                        long long row = -7;
                        const bool held = kfac::loss::take_row(s, n, stages, row);
                        check(held || (s.reads == 0 && row == -7), "used a stage whose wait ran out", n, stages, begin, last);
                        check(!held || (row == n && s.others), "went on without the row", n, stages, begin, last);
                        ++paths;
                    } while (c.next());
                }
    // The end of a run, after which no row is given to the stage: row n, or none, was the last.
    for (int stages = 2; stages <= 4; ++stages)
        for (long long n = 0; n < 4 * stages; ++n)
            for (int begin : {(int)CONSUMED, (int)GIVEN, (int)LANDED}) {
                Choices c;
                do {
                    c.at = 0;
                    Stage s{c, n, stages, begin, begin == CONSUMED ? CONSUMED : LANDED};
                    const bool drained = kfac::loss::drain_stage(s, stages);
                    check(drained && s.event == s.last, "left with bytes on their way", n, stages, begin, s.last);
                    ++paths;
                } while (c.next());
            }
    std::printf("%lld orders, %d failures\n", paths, failures);
    return failures != 0;
}
