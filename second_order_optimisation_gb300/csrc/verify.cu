// verify.cu -- drafted tokens accepted or replaced (kfac_verify_draft).
//
// Two launches.  The first takes the softmax's statistics (m, s = sum_j 2^((z_j - m) k),
// k = log2(e) / tau) of the policy's rows and, unless they are given, of the draft's; rows
// are split over CTAs where there are few.  The second walks each sequence to its first
// token that is not accepted, and takes that row's new token, argmax_j r_j / E_j, in one
// pass over the row (of policy, draft and noise), split over CTAs where there are few
// sequences; the last CTA of a sequence joins them.
//
// Bound by memory: every row of logits is read once, and one row of each sequence again.
// Each quotient is formed from fp32 probabilities (relative error about 1e-6); what
// accepts a token is compared in fp64.
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
    float4 *best;   // [seqs][pick_splits]: quotient of r, its index, of p, its index
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
                auto m = Elem<DT>::lowest();
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
// ln of a score's probability.
__device__ __forceinline__ double log_prob(float z, float m, float s, float tau) {
    return ((double)z - (double)m) / (double)tau - log((double)s);
}
__device__ __forceinline__ bool distribution(float s) { return s > 0.f && s <= F32_MAX; }

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

template <int DT>
__global__ void __launch_bounds__(PICK_THREADS) verify_pick_kernel(const __grid_constant__ Params P) {
    __shared__ Stat pol[PICK_WARPS], dra[PICK_WARPS];
    __shared__ int fate_of, at_of;
    __shared__ Best rs[PICK_WARPS], ps[PICK_WARPS];
    __shared__ bool last;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int seq = blockIdx.x / P.pick_splits, split = blockIdx.x % P.pick_splits;
    const long long r0 = row_at(P, seq), r1 = row_at(P, seq + 1);
    if (r1 <= r0) {
        if (split == 0 && tid == 0) P.accepted[seq] = 0;
        return;
    }
    const bool drafted = P.draft.z && !P.greedy;
    // the walk, eight rows at a time
    Stat p{}, q{};
    long long row = r0;
    int fate = ACCEPTED;
    for (; fate == ACCEPTED; row += PICK_WARPS) {
        if (row + warp < r1) {
            const long long i = row + warp;
            const Stat s = join(P.parts + i * P.splits, P.splits, P.target.k, lane);
            if (lane == 0) pol[warp] = s;
            if (drafted && i + 1 < r1) {
                Stat d;
                if (P.saved) d = Stat{P.saved[i].x, P.saved[i].y, NONE};
                else d = join(P.parts + (P.rows + i) * P.splits, P.splits, P.draft.k, lane);
                if (lane == 0) dra[warp] = d;
            }
        }
        __syncthreads();
        if (warp == 0) {
            const long long i = row + lane;
            const bool in = lane < PICK_WARPS && i < r1;
            int f = ACCEPTED, bits = 0;
            long long x = -1;
            double lp = 0.;
            if (in) {
                const Stat s = pol[lane];
                if (!distribution(s.s)) {
                    f = NOTHING;
                    bits = ERR_NONFINITE;
                } else if (i + 1 == r1) {
                    f = FROM_P;
                } else {
                    x = token_at(P, i);
                    const bool is = x >= 0 && x < P.vocab;
                    if (x >= P.vocab) bits = ERR_TARGET;
                    if (is) lp = log_prob(score<DT>(P.target, i, (int)x), s.m, s.s, P.target.tau);
                    if (P.greedy) {
                        if (x != s.index) f = FROM_P;
                    } else if (!is) {
                        f = FROM_P;
                    } else {
                        double ratio = exp(lp);
                        if (drafted) {
                            const Stat d = dra[lane];
                            if (!distribution(d.s)) {
                                f = FROM_P;
                                bits = ERR_NONFINITE;
                            } else {
                                // (q = 0 and p > 0: infinite; both 0: NaN, and not accepted)
                                ratio = exp(lp - log_prob(score<DT>(P.draft, i, (int)x), d.m, d.s, P.draft.tau));
                            }
                        }
                        if (f == ACCEPTED && !((double)P.uniform[i] < ratio)) f = FROM_R;
                    }
                }
            }
            const unsigned stops = __ballot_sync(ALL_LANES, in && f != ACCEPTED);
            const int at = stops ? __ffs(stops) - 1 : 32;
            if (split == 0 && in && lane < at) {  // (the token is what it was where out is tokens)
                put_token(P, i, (int)x);
                if (P.logp) P.logp[i] = (float)lp;
            }
            if (lane > at) bits = 0;
            bits = __reduce_or_sync(ALL_LANES, bits);
            if (stops ? lane == at : lane == 0) {
                fate_of = stops ? f : ACCEPTED;
                at_of = at;
                if (split == 0 && bits) atomicOr(P.err, bits);
            }
        }
        __syncthreads();
        fate = fate_of;
        if (fate != ACCEPTED) {
            p = pol[at_of];
            q = dra[at_of];
            row += at_of - PICK_WARPS;  // (the loop's step)
        }
        __syncthreads();
    }
    if (!P.greedy) {
        // this CTA's part of the new token's row
        Best br{0.f, NONE}, bp{0.f, NONE};
        if (fate == FROM_R || fate == FROM_P) {
            const int per = (P.vocab + P.pick_splits - 1) / P.pick_splits;
            const int j0 = split * per, j1 = min(P.vocab, j0 + per);
            using bits = typename Elem<DT>::bits;
            const bits *zp = (const bits *)(P.target.z + row * P.target.ld_bytes);
            const bits *zq = (const bits *)(P.draft.z + row * P.draft.ld_bytes);
            const float *E = P.noise + seq * P.ld_noise;
            const float ip = 1.f / p.s, iq = 1.f / q.s;
            const bool residual = fate == FROM_R;
            const long long x = residual && !drafted ? token_at(P, row) : -1;
            for (int j = j0 + tid; j < j1; j += PICK_THREADS) {
                const float e = fmaxf(E[j], 1.17549435e-38f);
                const float a = ex2((Elem<DT>::value(zp[j]) - p.m) * P.target.k) * ip;
                if (a > 0.f) bp.take(a / e, j);
                if (residual) {
                    const float b = drafted ? ex2((Elem<DT>::value(zq[j]) - q.m) * P.draft.k) * iq : j == x ? a : 0.f;
                    if (a > b) br.take((a - b) / e, j);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float kr = __shfl_xor_sync(ALL_LANES, br.key, o), kp = __shfl_xor_sync(ALL_LANES, bp.key, o);
            const int jr = __shfl_xor_sync(ALL_LANES, br.at, o), jp = __shfl_xor_sync(ALL_LANES, bp.at, o);
            br.take(kr, jr);
            bp.take(kp, jp);
        }
        if (lane == 0) {
            rs[warp] = br;
            ps[warp] = bp;
        }
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < PICK_WARPS; ++w) {
                br.take(rs[w].key, rs[w].at);
                bp.take(ps[w].key, ps[w].at);
            }
            P.best[blockIdx.x] = make_float4(br.key, __int_as_float(br.at), bp.key, __int_as_float(bp.at));
            __threadfence();
            last = atomicAdd(&P.done[seq], 1u) == P.pick_splits - 1;
            __threadfence();
        }
        __syncthreads();
        if (!last) return;
    }
    if (warp == 0) {
        int token = -1;
        if (P.greedy) {
            if (fate != NOTHING) token = p.index;
        } else if (fate != NOTHING) {
            Best br{0.f, NONE}, bp{0.f, NONE};
            for (int i = lane; i < P.pick_splits; i += 32) {
                const float4 b = __ldcg(P.best + (long long)seq * P.pick_splits + i);
                br.take(b.x, __float_as_int(b.y));
                bp.take(b.z, __float_as_int(b.w));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float kr = __shfl_xor_sync(ALL_LANES, br.key, o), kp = __shfl_xor_sync(ALL_LANES, bp.key, o);
                const int jr = __shfl_xor_sync(ALL_LANES, br.at, o), jp = __shfl_xor_sync(ALL_LANES, bp.at, o);
                br.take(kr, jr);
                bp.take(kp, jp);
            }
            token = br.at != NONE ? br.at : bp.at;
        }
        if (lane == 0) {
            P.accepted[seq] = (int)(row - r0);
            put_token(P, row, token);
            if (P.logp)
                P.logp[row] = token < 0 ? __int_as_float(0x7fc00000)
                                        : (float)log_prob(score<DT>(P.target, row, token), p.m, p.s, P.target.tau);
        }
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
    if (!d->greedy) {
        if (d->rows > 0 && (!d->uniform || !d->noise || d->ld_noise < d->vocab)) return KFAC_ERR_INVALID;
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
    P.best = ws.take<float4>((size_t)d.seqs * s.pick);
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
    if (!all_on_this_device({d.logits, d.tokens, d.seq_offsets, d.accepted, d.out_tokens, d.logp}) ||
        (draws && !all_on_this_device({d.draft, d.draft_saved, d.uniform, d.noise})))
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
