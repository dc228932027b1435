// loss.cu -- the entry points of the losses on logits (kernels: loss.cuh) and the
// kernels that see no logits: the policy loss's table of rows, and the pairs of the
// preference loss.
#include "loss.cuh"

namespace kfac {
namespace loss {

KFAC_LOSS_LAUNCHES(extern, KFAC_BF16)
KFAC_LOSS_LAUNCHES(extern, KFAC_F16)
KFAC_LOSS_LAUNCHES(extern, KFAC_F32)

namespace {

#define KFAC_BY_TYPE(dtype, launch, ...)                     \
    ((dtype) == KFAC_BF16  ? launch<KFAC_BF16>(__VA_ARGS__)  \
     : (dtype) == KFAC_F16 ? launch<KFAC_F16>(__VA_ARGS__)   \
                           : launch<KFAC_F32>(__VA_ARGS__))
kfac_status rows_run(int dtype, const RowParams &P, bool ent, cudaStream_t st) {
    return KFAC_BY_TYPE(dtype, launch_rows, P, ent, st);
}
kfac_status grad_run(int dtype, const GradParams &P, bool ent, cudaStream_t st) {
    return KFAC_BY_TYPE(dtype, launch_grad, P, ent, st);
}

// One cluster of CTAs, each a run of rows: every row's target, weight, advantage
// and old log-probability in one place, and the rows that are not ignored before
// the ignored ones, so that CTAs that stride over them get equal shares (where the ring
// takes them).  Bound by the latency of its few dependent loads, four rows to a thread
// at once: 16391 rows take 14 us, 60000 without the order 22 (33 with it, one at a time).
__global__ void __launch_bounds__(ROWS_THREADS) policy_rows_kernel(const __grid_constant__ PolicyRows P) {
    __shared__ int part[32], live_of[SMALL_CLUSTER], bad_of[SMALL_CLUSTER], warp_live[ROWS_THREADS / 32];
    cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid % 32, rank = blockIdx.x, ctas = gridDim.x;
    const long long per = (P.rows + ctas - 1) / ctas, r0 = min(P.rows, rank * per), r1 = min(P.rows, r0 + per);
    int n = 0, bad = 0;
    constexpr int BATCH = 4;
    for (long long base = r0 + tid; base < r1; base += BATCH * ROWS_THREADS) {
        PolicyRow q[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            q[i].target = -1;
            if (base + i * ROWS_THREADS < r1) q[i] = policy_row(P, base + i * ROWS_THREADS, bad);
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            n += q[i].target >= 0;
            if (base + i * ROWS_THREADS < r1) P.meta[base + i * ROWS_THREADS] = q[i];
        }
    }
    n = block_sum(n, part);
    bad = block_sum(bad, part);
    cluster_wait();
    if (tid < ctas) {
        *peer(&live_of[rank], tid) = n;
        *peer(&bad_of[rank], tid) = bad;
    }
    cluster_sync();
    int live = 0, before = 0, any = 0;
    for (int i = 0; i < ctas; ++i) {
        live += live_of[i];
        if (i < rank) before += live_of[i];
        any += bad_of[i];
    }
    if (rank == 0 && tid == 0) {
        *P.err = any ? ERR_TARGET : 0;
        *P.done = 0;
    }
    // (a CTA writes what its own threads have written, so its own barriers order it)
    const float w = 1.f / (float)live;
    const bool equal = !P.weight && !P.seq_mean;
    for (long long row = r0 + tid; !P.order && equal && row < r1; row += ROWS_THREADS)
        if (P.meta[row].target >= 0) P.meta[row].weight = w;
    for (long long base = r0; P.order && base < r1; base += ROWS_THREADS) {
        const long long row = base + tid;
        const bool in = row < r1, is = in && P.meta[row].target >= 0;
        const unsigned votes = __ballot_sync(0xffffffffu, is);
        __syncthreads();
        if (lane == 0) warp_live[tid / 32] = __popc(votes);
        __syncthreads();
        int mine = before + __popc(votes & ((1u << lane) - 1)), tile = 0;
        for (int i = 0; i < ROWS_THREADS / 32; ++i) {
            if (i < tid / 32) mine += warp_live[i];
            tile += warp_live[i];
        }
        // ignored rows so far: all rows before this one less the live ones before it
        if (in) P.order[is ? mine : live + (row - mine)] = (int)row;
        if (is && equal) P.meta[row].weight = w;
        before += tile;
    }
    if (!P.seq_mean) return;
    cluster_sync();  // the other CTAs' rows
    for (int q = rank * (ROWS_THREADS / 32) + tid / 32; q < P.seqs; q += ctas * (ROWS_THREADS / 32)) {
        const long long q0 = clamp_row(P.off[q], P.rows), q1 = clamp_row(P.off[q + 1], P.rows);
        int c = 0;
        for (long long row = q0 + lane; row < q1; row += 32) c += __ldcg(&P.meta[row].target) >= 0;
        c = __reduce_add_sync(0xffffffffu, c);
        for (long long row = q0 + lane; row < q1; row += 32)
            if (__ldcg(&P.meta[row].target) >= 0) P.meta[row].weight = 1.f / ((float)P.seqs * (float)c);
    }
}

// A CTA to each pair; the last to finish adds up the loss.  Bound by the
// latency of a chain of dependent loads and two reductions, 6 to 12 us.
__global__ void __launch_bounds__(PAIR_THREADS) pref_pairs_kernel(const __grid_constant__ PrefPairs P,
                                                                  const __grid_constant__ PrefSum U) {
    __shared__ bool last;
    pdl_wait();
    pdl_trigger();
    pref_pair<PAIR_THREADS>(P, blockIdx.x);
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(U.done, 1u) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (last) pref_sum(U);
}

size_t elem_size(int dtype) { return dtype == KFAC_F32 ? 4 : 2; }

// The arguments that every call on logits shares.
kfac_status check_logits(int dtype, const void *logits, long long ld, long long rows, int vocab, const void *target,
                         float tau) {
    if (dtype != KFAC_BF16 && dtype != KFAC_F16 && dtype != KFAC_F32) return KFAC_ERR_INVALID;
    if (rows < 0 || vocab < 1 || ld < vocab || (rows > 0 && (!logits || !target))) return KFAC_ERR_INVALID;
    if ((uintptr_t)logits % elem_size(dtype)) return KFAC_ERR_INVALID;
    // (below about 4.2e-39 the factor of the exponents is infinite)
    if (!(tau > 0.f) || !std::isfinite(tau) || !std::isfinite(LOG2E / tau)) return KFAC_ERR_INVALID;
    if (vocab > (1 << 24) || rows > 0x7fffffffLL) return KFAC_ERR_UNSUPPORTED;
    return KFAC_OK;
}
bool bad_grad(int dtype, const void *d, long long ld_d, int vocab) {
    return d && (ld_d < vocab || (uintptr_t)d % elem_size(dtype));
}

template <class D>
LogitsIn logits_in(const D &d) {
    return LogitsIn{(const char *)d.logits, d.ld * (long long)elem_size(d.dtype), d.target, d.target_i32, d.vocab,
                    d.temperature, LOG2E / d.temperature};
}

// ------------------------------------------------------------ policy loss

kfac_status check_policy(const kfac_policy_desc *d) {
    if (!d) return KFAC_ERR_INVALID;
    kfac_status s = check_logits(d->dtype, d->logits, d->ld, d->rows, d->vocab, d->target, d->temperature);
    if (s == KFAC_ERR_INVALID) return s;
    if (!d->stats || (d->rows > 0 && (!d->advantage || !d->old_logp)) || bad_grad(d->dtype, d->dlogits, d->ld_d, d->vocab))
        return KFAC_ERR_INVALID;
    if (!(d->clip_low >= 0.f) || !(d->clip_high >= 0.f) || !std::isfinite(d->kl_coef) ||
        !std::isfinite(d->entropy_coef) || !std::isfinite(d->grad_scale))
        return KFAC_ERR_INVALID;
    if ((d->seq_offsets && d->seqs < 1) || (d->seq_mean && (!d->seq_offsets || d->weight))) return KFAC_ERR_INVALID;
    if ((d->kl_coef != 0.f || d->kl) && !d->ref_logp) return KFAC_ERR_INVALID;
    return s;
}

struct PolicyPlan {
    int *err;
    PolicyRow *meta;
    int *order;
    TermSums *sums;
    unsigned *done;
    float2 *ms, *g;  // ms, g, h: for rows that do not fit the chip
    float *h;
};
// Whether the rows' launch is the ring, which takes the live rows first.
bool in_order(const kfac_policy_desc &d) {
    const long long whole = d.vocab / (d.dtype == KFAC_F32 ? 4 : 8);
    return d.dlogits && !by_warps(whole, d.rows, true) && ring_of(d.dtype, d.vocab, d.rows).cs;
}
// Whether one launch makes statistics and gradient.
bool rows_kept(const kfac_policy_desc &d) {
    const long long whole = d.vocab / (d.dtype == KFAC_F32 ? 4 : 8);
    return by_warps(whole, d.rows, d.dlogits) || ring_of(d.dtype, d.vocab, d.rows).cs;
}
PolicyPlan plan_policy(const kfac_policy_desc &d, Arena &ws) {
    PolicyPlan p{};
    const size_t n = (size_t)d.rows;
    p.err = ws.take<int>(64);
    p.meta = ws.take<PolicyRow>(n);
    if (in_order(d)) p.order = ws.take<int>(n);
    p.sums = ws.take<TermSums>(std::min<size_t>(n, MAX_CTAS));
    p.done = ws.take<unsigned>(1);
    if (!rows_kept(d)) {
        p.ms = ws.take<float2>(n);
        p.g = ws.take<float2>(n);
        p.h = ws.take<float>(n);
    }
    return p;
}

// ------------------------------------------------------------ preference loss

kfac_status check_preference(const kfac_preference_desc *d) {
    if (!d) return KFAC_ERR_INVALID;
    kfac_status s = check_logits(d->dtype, d->logits, d->ld, d->rows, d->vocab, d->target, d->temperature);
    if (s == KFAC_ERR_INVALID) return s;
    if (!d->seq_offsets || !d->loss || d->pairs < 1 || bad_grad(d->dtype, d->dlogits, d->ld_d, d->vocab))
        return KFAC_ERR_INVALID;
    if (d->kind != KFAC_PREF_SIGMOID && d->kind != KFAC_PREF_HINGE && d->kind != KFAC_PREF_IPO) return KFAC_ERR_INVALID;
    if (!(d->beta > 0.f) || !std::isfinite(d->beta) || !std::isfinite(d->grad_scale)) return KFAC_ERR_INVALID;
    if (!(d->label_smoothing >= 0.f) || !(d->label_smoothing < 1.f) ||
        (d->label_smoothing != 0.f && d->kind != KFAC_PREF_SIGMOID))
        return KFAC_ERR_INVALID;
    if (d->pairs > 0x3fffffff) return KFAC_ERR_UNSUPPORTED;
    return s;
}

struct PrefPlan {
    int *err, *bad;
    unsigned *done;
    float *logp, *row_g;
    float2 *ms;
    float *terms;
};
PrefPlan plan_preference(const kfac_preference_desc &d, Arena &ws) {
    PrefPlan p;
    const size_t n = (size_t)d.rows;
    p.err = ws.take<int>(64);
    p.done = ws.take<unsigned>(1);
    p.logp = ws.take<float>(n);
    p.row_g = ws.take<float>(n);
    p.ms = ws.take<float2>(n);
    p.terms = ws.take<float>((size_t)d.pairs);
    p.bad = ws.take<int>((size_t)d.pairs);
    return p;
}

}  // namespace
}  // namespace loss
}  // namespace kfac

using namespace kfac;
using namespace kfac::loss;

extern "C" kfac_status kfac_token_logprob(const kfac_logprob_desc *desc, void *stream) {
    if (!desc) return KFAC_ERR_INVALID;
    const kfac_logprob_desc &d = *desc;
    kfac_status s = check_logits(d.dtype, d.logits, d.ld, d.rows, d.vocab, d.target, d.temperature);
    if (s != KFAC_OK) return s;
    if (d.rows == 0) return KFAC_OK;
    if (!d.logp || (uintptr_t)d.saved % 8) return KFAC_ERR_INVALID;
    if (!all_on_this_device({d.logits, d.target, d.logp, d.lse, d.entropy, d.saved})) return KFAC_ERR_INVALID;
    RowParams P{};
    P.in = logits_in(d);
    P.rows = d.rows;
    P.nan_target = true;
    P.logp = d.logp;
    P.lse = d.lse;
    P.entropy = d.entropy;
    P.ms = (float2 *)d.saved;
    return rows_run(d.dtype, P, d.entropy != nullptr, (cudaStream_t)stream);
}

extern "C" kfac_status kfac_token_logprob_grad(const kfac_logprob_grad_desc *desc, void *stream) {
    if (!desc) return KFAC_ERR_INVALID;
    const kfac_logprob_grad_desc &d = *desc;
    kfac_status s = check_logits(d.dtype, d.logits, d.ld, d.rows, d.vocab, d.target, d.temperature);
    if (s == KFAC_ERR_INVALID) return s;
    if ((d.rows > 0 && (!d.saved || !d.dlogp || !d.dlogits)) || (d.dentropy && !d.entropy) || (uintptr_t)d.saved % 8 ||
        bad_grad(d.dtype, d.dlogits, d.ld_d, d.vocab))
        return KFAC_ERR_INVALID;
    if (s != KFAC_OK || d.rows == 0) return s;
    if (!all_on_this_device({d.logits, d.target, d.saved, d.entropy, d.dlogp, d.dentropy, d.dlogits}))
        return KFAC_ERR_INVALID;
    GradParams P{logits_in(d), d.rows, (const float2 *)d.saved, d.entropy, d.dlogp, d.dentropy, 1,
                 1.f / d.temperature, (char *)d.dlogits, d.ld_d * (long long)elem_size(d.dtype)};
    return grad_run(d.dtype, P, d.dentropy != nullptr, (cudaStream_t)stream);
}

extern "C" size_t kfac_policy_loss_workspace_size(const kfac_policy_desc *desc) {
    if (check_policy(desc) != KFAC_OK) return 0;
    Arena a;
    plan_policy(*desc, a);
    return a.used;
}

extern "C" kfac_status kfac_policy_loss(const kfac_policy_desc *desc, void *workspace, size_t workspace_bytes,
                                        void *stream) {
    kfac_status s = check_policy(desc);
    if (s != KFAC_OK) return s;
    const kfac_policy_desc &d = *desc;
    if (!workspace || ((uintptr_t)workspace % 256) != 0) return KFAC_ERR_WORKSPACE;
    Arena ws(workspace, workspace_bytes);
    const PolicyPlan p = plan_policy(d, ws);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    if (!all_on_this_device({d.logits, d.target, d.advantage, d.old_logp, d.ref_logp, d.weight, d.seq_offsets,
                             d.stats, d.logp, d.kl, d.entropy, d.dlogits}))
        return KFAC_ERR_INVALID;
    cudaStream_t st = (cudaStream_t)stream;
    const LogitsIn in = logits_in(d);
    PolicyRows R{in, d.rows, d.weight, d.advantage, d.old_logp, d.seq_offsets, d.seqs, d.seq_mean, p.meta,
                 p.order, p.done, p.err};
    const bool kept = rows_kept(d), ent = d.entropy_coef != 0.f || d.entropy;
    const float scale = d.dlogits ? d.grad_scale / d.temperature : 1.f;
    RowParams P{};
    P.in = in;
    P.rows = d.rows;
    P.policy = true;
    P.logp = d.logp;
    P.entropy = d.entropy ? d.entropy : ent && !kept ? p.h : nullptr;
    P.ref_logp = d.ref_logp;
    P.clip_low = d.clip_low;
    P.clip_high = d.clip_high;
    P.kl_coef = d.kl_coef;
    P.entropy_coef = d.entropy_coef;
    P.kl = d.kl;
    P.scale = scale;
    if (kept) P.dlogits = (char *)d.dlogits;
    P.ld_d_bytes = d.ld_d * (long long)elem_size(d.dtype);
    if (const int L = d.rows == 0 ? 8 : d.seq_mean ? 0 : small_lanes(d.dtype, d.vocab, d.rows))
        return KFAC_BY_TYPE(d.dtype, launch_policy_small, P, R, d.stats, L, ent, st);
    const unsigned ctas = d.rows > ROWS_THREADS ? SMALL_CLUSTER : 1;
    KFAC_LAUNCH_CLUSTERS(KK_LOSS_SMALL, st, policy_rows_kernel, ctas, ctas, ROWS_THREADS, 0, R);
    P.meta = p.meta;
    P.order = p.order;
    P.sums = p.sums;
    P.done = p.done;
    P.stats = d.stats;
    P.ms = p.ms;
    P.g = p.g;
    P.err = p.err;
    if ((s = rows_run(d.dtype, P, ent, st)) != KFAC_OK) return s;
    if (kept || !d.dlogits) return KFAC_OK;
    GradParams G{in, d.rows, p.ms, d.entropy ? d.entropy : p.h, (const float *)p.g, (const float *)p.g + 1, 2, scale,
                 (char *)d.dlogits, d.ld_d * (long long)elem_size(d.dtype)};
    return grad_run(d.dtype, G, d.entropy_coef != 0.f, st);
}

extern "C" size_t kfac_preference_loss_workspace_size(const kfac_preference_desc *desc) {
    if (check_preference(desc) != KFAC_OK) return 0;
    Arena a;
    plan_preference(*desc, a);
    return a.used;
}

extern "C" kfac_status kfac_preference_loss(const kfac_preference_desc *desc, void *workspace, size_t workspace_bytes,
                                            void *stream) {
    kfac_status s = check_preference(desc);
    if (s != KFAC_OK) return s;
    const kfac_preference_desc &d = *desc;
    if (!workspace || ((uintptr_t)workspace % 256) != 0) return KFAC_ERR_WORKSPACE;
    Arena ws(workspace, workspace_bytes);
    const PrefPlan p = plan_preference(d, ws);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    if (!all_on_this_device({d.logits, d.target, d.seq_offsets, d.ref_logp, d.pair_weight, d.loss, d.pair_loss,
                             d.seq_logp, d.token_logp, d.dlogits}))
        return KFAC_ERR_INVALID;
    cudaStream_t st = (cudaStream_t)stream;
    float *logp = d.token_logp ? d.token_logp : p.logp;
    RowParams P{};
    P.in = logits_in(d);
    P.rows = d.rows;
    P.off = d.seq_offsets;
    P.last = 2 * d.pairs;
    P.logp = logp;
    P.ms = p.ms;
    P.zero = p.done;
    P.zero_g = p.row_g;
    P.scale = d.grad_scale / d.temperature;
    P.ld_d_bytes = d.ld_d * (long long)elem_size(d.dtype);
    PrefPairs Q{d.target, d.target_i32, d.vocab, d.rows, d.seq_offsets, d.pairs, d.ref_logp, d.pair_weight, d.kind,
                d.average, d.beta, d.label_smoothing, d.dlogits ? P.scale : 0.f, logp, p.ms, p.row_g, p.terms, p.bad, d.pair_loss, d.seq_logp};
    PrefSum U{p.terms, p.bad, d.pairs, d.loss, p.err, p.done};
    // (a warp goes over a pair's rows and, in turn, over few pairs)
    const int L = d.rows == 0 ? 8 : d.pairs <= SMALL_CLUSTER * ROWS_THREADS ? small_lanes(d.dtype, d.vocab, d.rows) : 0;
    if (L) return KFAC_BY_TYPE(d.dtype, launch_pref_small, P, Q, U, (char *)d.dlogits, L, st);
    if ((s = rows_run(d.dtype, P, false, st)) != KFAC_OK) return s;
    KFAC_LAUNCH(KK_LOSS_SMALL, st, pref_pairs_kernel, (unsigned)d.pairs, PAIR_THREADS, 0, Q, U);
    if (!d.dlogits) return KFAC_OK;
    GradParams G{logits_in(d), d.rows, p.ms, nullptr, p.row_g, nullptr, 1, P.scale, (char *)d.dlogits, P.ld_d_bytes};
    return grad_run(d.dtype, G, false, st);
}
