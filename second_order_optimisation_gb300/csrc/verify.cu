// verify.cu -- drafted tokens accepted or replaced (kfac_verify_draft).
//
// Two launches.  The first takes the softmax's statistics (m, s = sum_j 2^((z_j - m) k),
// k = log2(e) / tau) of the policy's rows and, unless they are given, of the draft's; rows
// are split over CTAs where there are few.  The second walks each sequence to its first
// token that is not accepted, and takes that row's new token, argmax_j r_j / E_j, in one
// pass over the row (of policy, draft and noise), split over CTAs where there are few
// sequences; the last CTA of a sequence joins them.  Rows behind a token that is not accepted are
// read too: ways that read only those needed (a cluster that goes through a sequence row by
// row; rows in three waves with a look at each sequence between them) took 283 and 208 us in place
// of 225 for 256 x 8 rows of 131072 of whose tokens 86% are accepted, and more for fewer rows.
//
// Bound by memory: every row of logits is read once, and one row of each sequence again.
// p and q are fp32 (relative error about 1e-6), so r = p - q is off by as much of the larger of
// the two: where policy and draft nearly agree, few of its bits are right.  What accepts a token is
// compared in fp64 where fp32's arithmetic on scores and sums could err; the sums themselves are
// fp32 (off by 1e-7 to 1e-6, the more the further a row's weight lies below its maximum).
#include <algorithm>
#include <cmath>

#include "logits.cuh"

namespace kfac {
namespace {

constexpr int STAT_THREADS = 128, BATCH = 4, PICK_THREADS = 256, PICK_WARPS = PICK_THREADS / 32;
constexpr int NONE = 0x7fffffff;

struct Scores {
    const char *z;
    long long ld_bytes;
    float k, tau;
};
struct Params {
    Scores target, draft;  // draft.z NULL: there is none
    const float2 *saved;   // of the draft's rows, or NULL
    long long rows;
    int vocab, seqs, token_i32, greedy;
    const int32_t *off;
    const void *tokens;
    const float *uniform, *noise;
    long long ld_noise;
    int32_t *accepted;
    void *out;
    float *logp;
    // scratch
    float4 *parts;  // [units][splits]: maximum, sum, its index (greedy)
    float2 *best;   // [seqs][pick_splits]: the largest quotient, its index
    unsigned *done; // [seqs]
    int *err;
    int splits, pick_splits;
};

__device__ __forceinline__ long long row_at(const Params &P, int i) {
    return min(max((long long)P.off[i], 0LL), P.rows);
}

// The lowest index with a value of M among elements of 16-byte groups.
template <int DT>
__device__ __forceinline__ int index_of(uint4 u, int first, int n, float M) {
    float v[Elem<DT>::N];
    Elem<DT>::unpack(u, v);
    int best = NONE;
#pragma unroll
    for (int i = Elem<DT>::N - 1; i >= 0; --i)
        if (v[i] == M && first + i >= 0 && first + i < n) best = first + i;
    return best;
}

template <int DT>
__global__ void __launch_bounds__(STAT_THREADS) verify_stats_kernel(const __grid_constant__ Params P) {
    constexpr int T = STAT_THREADS;
    __shared__ Part parts[T / 32];
    __shared__ int index;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        if (tid == 0) *P.err = 0;
        for (int i = tid; i < P.seqs; i += T) P.done[i] = 0;
    }
    const bool drafted = P.draft.z && !P.saved && !P.greedy;
    const long long units = P.rows * (drafted ? 2 : 1);
    for (long long item = blockIdx.x; item < units * P.splits; item += gridDim.x) {
        const long long unit = item / P.splits;
        const int split = (int)(item % P.splits);
        const bool of_draft = unit >= P.rows;
        const long long row = of_draft ? unit - P.rows : unit;
        const Scores &S = of_draft ? P.draft : P.target;
        if (of_draft) {  // no token was drawn from the row behind the drafted ones
            bool last = false;
            for (int i = tid; i < P.seqs; i += T) last |= row_at(P, i + 1) == row + 1 && row_at(P, i) <= row;
            if (__syncthreads_or(last)) continue;
        }
        const Row<DT> r(S.z + row * S.ld_bytes, P.vocab);
        const int per = (r.end() - r.begin() + P.splits - 1) / P.splits;
        const int c0 = r.begin() + split * per, g1 = min(r.end(), c0 + per);
        const int at = split != 0 ? -1 : tid == 0 && r.has_front() ? 0 : tid == 1 && r.has_back() ? r.end() : -1;
        Running<DT, false> run(S.k);
        float top = -INFINITY;  // (greedy) the largest of the batches so far, and the first batch that has it
        int top_at = -1;
        for (int g = c0 + tid; g - tid < g1; g += BATCH * T) {
            uint4 u[BATCH];
            const int most = min(BATCH, (g1 - (g - tid) + T - 1) / T);
            unsigned skip = 0;
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i < most) {
                    u[i] = r.load_whole(min(g + i * T, g1 - 1));
                    skip |= (g + i * T >= g1 ? 1u : 0u) << i;
                }
            run.template add<BATCH>(u, most, skip);
            if (P.greedy) {
                auto m = Elem<DT>::nothing();  // (not the lowest finite value: a batch of masked scores does not hold it)
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
                    if (i < most) m = Elem<DT>::raise(m, u[i]);
                if (Elem<DT>::largest(m) > top) {
                    top = Elem<DT>::largest(m);
                    top_at = g;
                }
            }
        }
        uint4 edge = Row<DT>::none();
        if (at >= 0) {
            edge = r.load_edge(at);
            run.template add<1>(&edge, 1, 0);
        }
        const Part mine = run.part();
        if (tid % 32 == 0) parts[tid / 32] = mine;
        if (tid == 0) index = NONE;
        __syncthreads();
        float M = parts[0].m;
#pragma unroll
        for (int w = 1; w < T / 32; ++w) M = fmaxf(M, parts[w].m);
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < T / 32; ++w) s += relative_to<false>(parts[w], M, S.k).s;
        if (P.greedy) {
            int found = NONE;
            if (top == M)  // (a thread's groups past the end are the last one again)
                for (int i = 0; i < BATCH; ++i) {
                    const int g = top_at + i * T;
                    if (g < g1) found = min(found, index_of<DT>(r.load_whole(g), r.first(g), r.n, M));
                }
            if (at >= 0) found = min(found, index_of<DT>(edge, r.first(at), r.n, M));
            if (found != NONE) atomicMin(&index, found);
            __syncthreads();
        }
        if (tid == 0) P.parts[item] = make_float4(M, s, __int_as_float(index), 0.f);
        __syncthreads();
    }
}

struct Stat {
    float m, s;
    int index;
};
// A row's parts joined by a warp; on every lane.
__device__ __forceinline__ Stat join(const float4 *parts, int splits, float k, int lane) {
    float m = -F32_MAX;
    float4 p[2];
    int n = 0;
    float s = 0.f;
    int index = NONE;
    // (the maximum first, then the sums: the parts are in L1 or L2 the second time)
    for (int i = lane; i < splits; i += 32) {
        const float4 q = __ldcg(parts + i);
        if (n < 2) p[n++] = q;
        m = fmaxf(m, q.x);
    }
    m = lanes_max(m, 32);
    for (int i = lane, j = 0; i < splits; i += 32, ++j) {
        const float4 q = j < 2 ? p[j] : __ldcg(parts + i);
        s += relative_to<false>(Part{q.x, q.y, 0.f}, m, k).s;
        if (q.x == m) index = min(index, __float_as_int(q.z));
    }
    Stat r;
    r.m = m;
    r.s = lanes_sum(s, 32);
    r.index = __reduce_min_sync(ALL_LANES, index);
    return r;
}

__device__ __forceinline__ long long token_at(const Params &P, long long row) {
    return P.token_i32 ? ((const int32_t *)P.tokens)[row] : ((const int64_t *)P.tokens)[row];
}
__device__ __forceinline__ void put_token(const Params &P, long long row, int t) {
    if (P.token_i32) ((int32_t *)P.out)[row] = t;
    else ((int64_t *)P.out)[row] = t;
}
template <int DT>
__device__ __forceinline__ float score(const Scores &S, long long row, int j) {
    return Elem<DT>::value(((const typename Elem<DT>::bits *)(S.z + row * S.ld_bytes))[j]);
}
__device__ __forceinline__ bool distribution(float s) { return s > 0.f && s <= F32_MAX; }
__device__ __forceinline__ float log_prob(float z, const Stat &s, float tau) {
    return (z - s.m) / tau - LN2 * log2f(s.s);
}
// Whether u < p / q.  In fp32 where the two are further apart than its error, else in fp64 from the same
// sums: then as right as these are.
__device__ __noinline__ bool below_exact(float u, float zp, Stat p, float taup, float zq, Stat q, float tauq) {
    const double lp = ((double)zp - (double)p.m) / (double)taup - log((double)p.s);
    const double lq = q.s > 0.f ? ((double)zq - (double)q.m) / (double)tauq - log((double)q.s) : 0.;
    return (double)u < exp(lp - lq);  // (q = 0: infinite where p > 0; both 0: NaN, not below)
}
// q.s = 0: a token that was not drawn, q = 1.
__device__ __forceinline__ bool below_ratio(float u, float zp, const Stat &p, const Scores &P, float zq, const Stat &q,
                                            const Scores &Q) {
    const float yp = (zp - p.m) * P.k, yq = q.s > 0.f ? (zq - q.m) * Q.k : 0.f;
    const float ratio = exp2f((yp - log2f(p.s)) - (q.s > 0.f ? yq - log2f(q.s) : 0.f));
    const float off = 1e-5f + 4e-7f * (fabsf(yp) + fabsf(yq));
    if (u < ratio * (1.f - off)) return true;
    if (u > ratio * (1.f + off)) return false;
    return below_exact(u, zp, p, P.tau, zq, q, Q.tau);
}

// What became of a row: its token accepted; replaced by a draw from r, or from p; or no
// distribution to draw from.
enum Fate : int { ACCEPTED = 0, FROM_R = 1, FROM_P = 2, NOTHING = 3 };

struct Best {
    float key;
    int at;
    __device__ __forceinline__ void take(float k, int j) {
        if (k > key || (k == key && j < at)) {
            key = k;
            at = j;
        }
    }
};
__device__ __forceinline__ Best best_of_warp(Best b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float k = __shfl_xor_sync(ALL_LANES, b.key, o);
        const int j = __shfl_xor_sync(ALL_LANES, b.at, o);
        b.take(k, j);
    }
    return b;
}
// On every thread of warp 0.
__device__ __forceinline__ Best best_of_block(Best b, Best *shared) {
    b = best_of_warp(b);
    if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = b;
    __syncthreads();
    return best_of_warp(threadIdx.x % 32 < PICK_WARPS ? shared[threadIdx.x % 32] : Best{0.f, NONE});
}

// A row's probabilities, of which one is drawn: p, or r = max(p - q, 0).
struct Row2 {
    Stat p, q;
    float lp, lq;  // log2 of the sums
    float kp, kq;
    long long x;   // FROM_R of a token that was not drawn: the token (q = 1 there)
    bool drafted;
    __device__ __forceinline__ float value(float zp, float zq) const {
        const float a = ex2(fmaf(zp - p.m, kp, -lp));
        return drafted ? a - ex2(fmaf(zq - q.m, kq, -lq)) : a;
    }
    __device__ __forceinline__ void take(Best &b, float v, float e, int j) const {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaxf(e, 1.17549435e-38f)));
        const float key = v * inv;
        if (key > b.key && j != x) {
            b.key = key;
            b.at = j;
        }
    }
};

// The part of a row from a group on, with its noise: 16-byte groups of the policy's scores, the
// draft's at the same alignment, the noise at any.
template <int DT, bool ANY, bool DRAFTED>
__device__ __forceinline__ void race_groups(const Row2 &R, const Row<DT> &zp, const char *zq, const float *E, int g0, int g1,
                                            Best &best) {
    constexpr int N = Elem<DT>::N, STEP = PICK_THREADS, PER = 2;
    const int off = (int)((uintptr_t)(E + zp.first(g0)) & 15);
#pragma unroll 1
    for (int g = g0 + threadIdx.x; g < g1; g += PER * STEP) {
        uint4 u[PER], w[PER];
        Pieces<N / 4, ANY> e[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int h = min(g + i * STEP, g1 - 1);  // (the last group again where there is none)
            u[i] = zp.load_whole(h);
            if (DRAFTED) w[i] = ld16(zq + (size_t)h * 16);
            e[i].load((const char *)(E + zp.first(h)), off);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int h = min(g + i * STEP, g1 - 1);
            float a[N], b[N];
            uint4 f[N / 4];
            Elem<DT>::unpack(u[i], a);
            if (DRAFTED) Elem<DT>::unpack(w[i], b);
            e[i].take(off, f);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint32_t bits[4] = {f[j / 4].x, f[j / 4].y, f[j / 4].z, f[j / 4].w};
                R.take(best, R.value(a[j], DRAFTED ? b[j] : 0.f), __uint_as_float(bits[j % 4]), zp.first(h) + j);
            }
        }
    }
}
// The race over elements j0 .. j1 - 1 of a row; on every thread its own best.  By 16-byte groups
// where policy and draft lie alike (rows of one pitch do), else element by element: 256 rows
// of 131072 bf16 took 361 us element by element.
template <int DT>
__device__ __forceinline__ Best race(const Params &P, const Row2 &R, long long row, int seq, int j0, int j1) {
    using bits = typename Elem<DT>::bits;
    const char *p = P.target.z + row * P.target.ld_bytes, *q = P.draft.z + row * P.draft.ld_bytes;
    const float *E = P.noise + seq * P.ld_noise;
    Best b{0.f, NONE};
    auto one = [&](int j) {
        R.take(b, R.value(Elem<DT>::value(((const bits *)p)[j]), R.drafted ? Elem<DT>::value(((const bits *)q)[j]) : 0.f), E[j], j);
    };
    if (R.drafted && (((uintptr_t)p ^ (uintptr_t)q) & 15) != 0) {
#pragma unroll 4
        for (int j = j0 + threadIdx.x; j < j1; j += PICK_THREADS) one(j);
        return b;
    }
    // the groups that start in the part, and the row's edges
    const Row<DT> r(p, P.vocab);
    constexpr int N = Elem<DT>::N;
    const int g0 = max(r.begin(), (j0 + r.phase + N - 1) / N), g1 = min(r.end(), (j1 + r.phase + N - 1) / N);
    const int front = r.begin() * N - r.phase, back = r.end() * N - r.phase;  // first elements of the whole groups, and behind them
    if (j0 == 0 && (int)threadIdx.x < front && (int)threadIdx.x < P.vocab) one(threadIdx.x);
    if (g0 < g1) {
        const char *qb = R.drafted ? q - r.phase * (int)sizeof(bits) : nullptr;
        const bool any = ((uintptr_t)(E + r.first(g0)) & 15) != 0;
        if (R.drafted && any) race_groups<DT, true, true>(R, r, qb, E, g0, g1, b);
        else if (R.drafted) race_groups<DT, false, true>(R, r, qb, E, g0, g1, b);
        else if (any) race_groups<DT, true, false>(R, r, qb, E, g0, g1, b);
        else race_groups<DT, false, false>(R, r, qb, E, g0, g1, b);
    }
    if (j1 == P.vocab && back + (int)threadIdx.x < P.vocab && back >= front) one(back + threadIdx.x);
    return b;
}

template <int DT>
// 256 rows of 131072 bf16, draft and noise (268 MB, half of it in L2) take 57 us; two CTAs to an SM 67, four 66;
// the walk in a launch of its own and shorter parts of rows, 8 + 53.
__global__ void __launch_bounds__(PICK_THREADS, 3) verify_pick_kernel(const __grid_constant__ Params P) {
    __shared__ Stat pol[PICK_WARPS], dra[PICK_WARPS];
    __shared__ int fates[PICK_WARPS], flags[PICK_WARPS], new_token;
    __shared__ Best bests[PICK_WARPS];
    __shared__ bool last;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int seq = blockIdx.x / P.pick_splits, split = blockIdx.x % P.pick_splits;
    const int per = (P.vocab + P.pick_splits - 1) / P.pick_splits;
    const int j0 = min(P.vocab, split * per), j1 = min(P.vocab, j0 + per);
    // this part of the noise on its way to L2 while the sums are made (without rows there may be no noise)
    if (!P.greedy && P.rows > 0 && tid == 0 && j1 > j0) {
        const uintptr_t a = (uintptr_t)(P.noise + seq * P.ld_noise + j0) & ~(uintptr_t)15;
        const uintptr_t b = (uintptr_t)(P.noise + seq * P.ld_noise + j1) & ~(uintptr_t)15;
        if (b > a) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"((uint32_t)(b - a)) : "memory");
    }
    pdl_wait();
    pdl_trigger();
    const long long r0 = row_at(P, seq), r1 = row_at(P, seq + 1);
    if (r1 <= r0) {
        if (split == 0 && tid == 0) P.accepted[seq] = 0;
        return;
    }
    const bool drafted = P.draft.z && !P.greedy;
    // the walk, a row to a warp, eight at a time
    long long row = r0;
    int fate = ACCEPTED, at = 0;
    for (;; row += PICK_WARPS) {
        const long long i = row + warp;
        if (i < r1) {
            const bool bonus = i + 1 == r1;
            const long long x = bonus ? -1 : token_at(P, i);
            const bool is = x >= 0 && x < P.vocab;
            float zp = 0.f, zq = 0.f, u = 0.f;
            if (is) {
                zp = score<DT>(P.target, i, (int)x);
                if (drafted) zq = score<DT>(P.draft, i, (int)x);
                if (!P.greedy) u = P.uniform[i];
            }
            const Stat s = join(P.parts + i * P.splits, P.splits, P.target.k, lane);
            Stat d{0.f, 0.f, NONE};
            if (drafted && !bonus) {
                if (P.saved) d = Stat{P.saved[i].x, P.saved[i].y, NONE};
                else d = join(P.parts + (P.rows + i) * P.splits, P.splits, P.draft.k, lane);
            }
            int f = ACCEPTED, bits = !bonus && x >= P.vocab ? ERR_TARGET : 0;
            if (!distribution(s.s)) {
                f = NOTHING;
                bits = ERR_NONFINITE;
            } else if (P.greedy) {
                if (bonus || x != s.index) f = FROM_P;
            } else if (!is) {
                f = FROM_P;
            } else if (drafted && !distribution(d.s)) {
                f = FROM_P;
                bits = ERR_NONFINITE;
            } else if (!below_ratio(u, zp, s, P.target, zq, d, P.draft)) {
                f = FROM_R;
            }
            if (lane == 0) {
                pol[warp] = s;
                dra[warp] = d;
                fates[warp] = f;
                flags[warp] = bits;
            }
        }
        __syncthreads();
        const int n = (int)min((long long)PICK_WARPS, r1 - row);
        for (at = 0; at < n && fates[at] == ACCEPTED;) ++at;
        if (split == 0) {
            if (i < r1 && warp < at && lane == 0) {  // accepted (the token is what it was where out is tokens)
                const int x = (int)token_at(P, i);
                put_token(P, i, x);
                if (P.logp) P.logp[i] = log_prob(score<DT>(P.target, i, x), pol[warp], P.target.tau);
            }
            if (tid <= at && tid < n && flags[tid]) atomicOr(P.err, flags[tid]);
        }
        if (at < n) break;
        __syncthreads();
    }
    fate = fates[at];
    row += at;
    Row2 R;
    R.p = pol[at];
    R.q = dra[at];
    R.lp = log2f(R.p.s);
    R.kp = P.target.k;
    R.kq = P.draft.k;
    R.drafted = fate == FROM_R && drafted;
    R.lq = R.drafted ? log2f(R.q.s) : 0.f;
    R.x = fate == FROM_R && !drafted ? token_at(P, row) : -1;
    int token = -1;
    if (P.greedy) {
        if (fate != NOTHING) token = R.p.index;
    } else {
        // this CTA's part of the new token's row; the last CTA joins the parts
        Best b{0.f, NONE};
        if (fate != NOTHING) b = race<DT>(P, R, row, seq, j0, j1);
        b = best_of_block(b, bests);
        if (tid == 0) {
            P.best[blockIdx.x] = make_float2(b.key, __int_as_float(b.at));
            __threadfence();
            last = atomicAdd(&P.done[seq], 1u) == P.pick_splits - 1;
            __threadfence();
        }
        __syncthreads();
        if (!last) return;
        if (warp == 0) {
            Best all{0.f, NONE};
            for (int i = lane; i < P.pick_splits; i += 32) {
                const float2 c = __ldcg(P.best + (long long)seq * P.pick_splits + i);
                all.take(c.x, __float_as_int(c.y));
            }
            all = best_of_warp(all);
            if (lane == 0) new_token = all.at;
        }
        __syncthreads();
        token = new_token;
        if (token == NONE && fate == FROM_R) {  // r is nothing (p and q are equal): from p, by this CTA alone
            R.drafted = false;
            R.x = -1;
            b = race<DT>(P, R, row, seq, 0, P.vocab);
            __syncthreads();
            b = best_of_block(b, bests);
            if (tid == 0) new_token = b.at;
            __syncthreads();
            token = new_token;
        }
    }
    if (token == NONE) token = -1;
    if (tid == 0) {
        P.accepted[seq] = (int)(row - r0);
        put_token(P, row, token);
        if (P.logp)
            P.logp[row] = token < 0 ? __int_as_float(0x7fc00000) : log_prob(score<DT>(P.target, row, token), R.p, P.target.tau);
    }
    for (long long i = row + 1 + tid; i < r1; i += PICK_THREADS) {
        put_token(P, i, -1);
        if (P.logp) P.logp[i] = 0.f;
    }
}

size_t elem_size(int dtype) { return dtype == KFAC_F32 ? 4 : 2; }

bool bad_tau(float tau) { return !(tau > 0.f) || !std::isfinite(tau) || !std::isfinite(LOG2E / tau); }

kfac_status check(const kfac_verify_desc *d) {
    if (!d) return KFAC_ERR_INVALID;
    if (d->dtype != KFAC_BF16 && d->dtype != KFAC_F16 && d->dtype != KFAC_F32) return KFAC_ERR_INVALID;
    if (d->rows < 0 || d->seqs < 1 || d->vocab < 1 || d->ld < d->vocab || bad_tau(d->temperature)) return KFAC_ERR_INVALID;
    if (!d->seq_offsets || !d->accepted || (uintptr_t)d->logits % elem_size(d->dtype)) return KFAC_ERR_INVALID;
    if (d->rows > 0 && (!d->logits || !d->tokens || !d->out_tokens)) return KFAC_ERR_INVALID;
    if (((uintptr_t)d->tokens | (uintptr_t)d->out_tokens) % (d->token_i32 ? 4 : 8) ||
        ((uintptr_t)d->seq_offsets | (uintptr_t)d->accepted | (uintptr_t)d->logp) % 4)
        return KFAC_ERR_INVALID;
    if (!d->greedy) {
        if (d->rows > 0 && (!d->uniform || !d->noise || d->ld_noise < d->vocab)) return KFAC_ERR_INVALID;
        if (((uintptr_t)d->uniform | (uintptr_t)d->noise) % 4) return KFAC_ERR_INVALID;
        if (d->draft && (d->ld_draft < d->vocab || (uintptr_t)d->draft % elem_size(d->dtype) || bad_tau(d->draft_temperature)))
            return KFAC_ERR_INVALID;
        if (d->draft_saved && (!d->draft || (uintptr_t)d->draft_saved % 8)) return KFAC_ERR_INVALID;
    }
    if (d->vocab > (1 << 24) || d->rows > 0x7fffffffLL || d->seqs > (1 << 20)) return KFAC_ERR_UNSUPPORTED;
    return KFAC_OK;
}

struct Split {
    long long units;
    int stats, pick;
};
Split split_of(const kfac_verify_desc &d) {
    Split s;
    s.units = d.rows * (d.draft && !d.draft_saved && !d.greedy ? 2 : 1);
    const long long sms = device_sm_count();
    // CTAs for eight to an SM, a batch of loads at least to each thread of them
    const long long groups = std::max<long long>(1, d.vocab / (16 / (long long)elem_size(d.dtype)));
    s.stats = (int)std::max<long long>(1, std::min(ceil_div(8 * sms, std::max<long long>(s.units, 1)), groups / (STAT_THREADS * BATCH)));
    // for four to an SM, eight values at least to each thread
    s.pick = d.greedy ? 1 : (int)std::max<long long>(1, std::min(ceil_div(4 * sms, d.seqs), (long long)d.vocab / (8 * PICK_THREADS)));
    return s;
}

void plan(const kfac_verify_desc &d, Arena &ws, Params &P) {
    const Split s = split_of(d);
    P.splits = s.stats;
    P.pick_splits = s.pick;
    P.err = ws.take<int>(64);
    P.parts = ws.take<float4>((size_t)s.units * s.stats);
    P.best = ws.take<float2>((size_t)d.seqs * s.pick);
    P.done = ws.take<unsigned>((size_t)d.seqs);
}

template <int DT>
kfac_status launch(const Params &P, const kfac_verify_desc &d, cudaStream_t st) {
    const long long items = split_of(d).units * P.splits;
    const unsigned grid = (unsigned)std::max<long long>(1, std::min<long long>(items, 16LL * device_sm_count()));
    KFAC_LAUNCH(KK_VERIFY, st, verify_stats_kernel<DT>, grid, STAT_THREADS, 0, P);
    KFAC_LAUNCH(KK_VERIFY, st, verify_pick_kernel<DT>, (unsigned)(d.seqs * P.pick_splits), PICK_THREADS, 0, P);
    return KFAC_OK;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" size_t kfac_verify_draft_workspace_size(const kfac_verify_desc *desc) {
    if (check(desc) != KFAC_OK) return 0;
    Arena a;
    Params P{};
    plan(*desc, a, P);
    return a.used;
}

extern "C" kfac_status kfac_verify_draft(const kfac_verify_desc *desc, void *workspace, size_t workspace_bytes,
                                         void *stream) {
    const kfac_status s = check(desc);
    if (s != KFAC_OK) return s;
    const kfac_verify_desc &d = *desc;
    if (!workspace || ((uintptr_t)workspace % 256) != 0) return KFAC_ERR_WORKSPACE;
    Arena ws(workspace, workspace_bytes);
    Params P{};
    plan(d, ws, P);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    const bool draws = !d.greedy;
    DeviceMemory memory;
    if (!memory.holds_all({d.logits, d.tokens, d.seq_offsets, d.accepted, d.out_tokens, d.logp}) ||
        (draws && !memory.holds_all({d.draft, d.draft_saved, d.uniform, d.noise})))
        return KFAC_ERR_INVALID;
    const long long e = (long long)elem_size(d.dtype);
    P.target = Scores{(const char *)d.logits, d.ld * e, LOG2E / d.temperature, d.temperature};
    if (draws && d.draft) {
        P.draft = Scores{(const char *)d.draft, d.ld_draft * e, LOG2E / d.draft_temperature, d.draft_temperature};
        P.saved = (const float2 *)d.draft_saved;
    }
    P.rows = d.rows;
    P.vocab = d.vocab;
    P.seqs = d.seqs;
    P.token_i32 = d.token_i32;
    P.greedy = d.greedy;
    P.off = d.seq_offsets;
    P.tokens = d.tokens;
    P.uniform = d.uniform;
    P.noise = d.noise;
    P.ld_noise = d.ld_noise;
    P.accepted = d.accepted;
    P.out = d.out_tokens;
    P.logp = d.logp;
    cudaStream_t st = (cudaStream_t)stream;
    if (d.dtype == KFAC_BF16) return launch<KFAC_BF16>(P, d, st);
    if (d.dtype == KFAC_F16) return launch<KFAC_F16>(P, d, st);
    return launch<KFAC_F32>(P, d, st);
}
