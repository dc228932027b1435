// ring.h -- how a stage of the policy loss's ring is handed from the warp that
// fetches rows to the team that takes them: the order of the waits, apart from
// the instructions that make them, so that a host test can go through it with a
// model of the barriers.
//
// A stage has a barrier `full` (one phase for each row that it holds, complete
// when the row's bytes and other inputs are there) and a word `given`, the number
// of the row that it was given to last.  A wait on the barrier tells phases apart
// by their parity only, and so says something only about a phase that is the
// current one or the one before it.
#pragma once

#ifdef __CUDACC__
#define KFAC_RING_FN __host__ __device__ __forceinline__
#else
#define KFAC_RING_FN inline
#endif

namespace kfac {
namespace loss {

// The parity of row n's phase of its stage's barrier.
KFAC_RING_FN int stage_parity(long long n, int stages) { return (int)(n / stages & 1); }

// Waits until the stage holds row n; false when a wait runs out.  `given` comes
// first: while the stage is still another row's, that row's phase has the other
// parity, and a wait for row n's would pass at once, whatever becomes of the stage
// next.  Once the stage has been given to row n, its phase is the current one.
template <class Stage>
KFAC_RING_FN bool wait_stage(Stage &s, long long n, int stages) {
    if (s.given() != n) {
        s.start();
        while (s.given() != n)
            if (s.late()) return false;
    }
    return s.wait_full(stage_parity(n, stages));
}

// Row n's inputs besides its logits, into `row`, once the stage holds it.  False when
// the wait ran out for any thread of the warp: `row` is then as it was, and nothing of
// the stage (whose row may be another one, or none yet) may be used, so that no address
// is ever made from it.
template <class Stage, class Row>
KFAC_RING_FN bool take_row(Stage &s, long long n, int stages, Row &row) {
    if (!s.all(wait_stage(s, n, stages))) return false;
    row = s.row();
    return true;
}

// Waits until nothing is on its way into the stage any more: the phase of the row that
// it was given to last is complete.  (A wait on the other parity passes at once while
// that row's bytes are still coming.)
template <class Stage>
KFAC_RING_FN bool drain_stage(Stage &s, int stages) {
    const long long n = s.given();
    return n < 0 || s.wait_full(stage_parity(n, stages));
}

}  // namespace loss
}  // namespace kfac
