// loss.cu -- losses on logits: token log-probabilities and their gradient, the
// clipped policy loss with a KL term, and the preference loss over pairs.
//
// With y_j = (z_j - m) k, k = log2(e) / tau and m the row's maximum,
//   s = sum_j 2^y_j,  t = sum_j 2^y_j y_j,
//   logp = (z_target - m) / tau - ln s,   lse = m / tau + ln s,
//   H = ln 2 (log2 s - t / s),
// and the gradient of g logp + gh H (times the call's scale, over tau) is
//   d_j = 2^y_j (a + b y_j) + g [j = target],
//   b = - gh ln 2 / s,   a = - (g + gh (H - ln 2 log2 s)) / s.
// The maximum is subtracted before the scaling, so that rows whose logits are
// all the type's lowest value stay finite.
#include <cmath>

#include "logits.cuh"

namespace kfac {
namespace {

constexpr int THREADS = 256;

// What every row kernel reads.
struct LogitsIn {
    const char *logits;
    long long ld_bytes;
    const void *target;
    int target_i32;
    int vocab;
    float tau, k;  // k = log2(e) / tau
};

__device__ __forceinline__ long long target_of(const LogitsIn &in, long long row) {
    return in.target_i32 ? ((const int32_t *)in.target)[row] : ((const int64_t *)in.target)[row];
}

template <int DT>
__device__ __forceinline__ float logit_at(const void *row, long long j) {
    return Elem<DT>::value(((const typename Elem<DT>::bits *)row)[j]);
}

// A row's statistics as its log-probability, lse and entropy.  s = 0: every logit is -inf.
struct RowResult {
    float logp, lse, h;
};
__device__ __forceinline__ RowResult row_result(float m, float s, float t, float z_t, float tau) {
    RowResult r;
    if (s == 0.f) {
        r.logp = r.lse = -INFINITY;
        r.h = 0.f;
        return r;
    }
    const float l2 = log2f(s);
    r.logp = (z_t - m) / tau - LN2 * l2;
    r.lse = m / tau + LN2 * l2;
    r.h = LN2 * (l2 - t / s);
    return r;
}

// ------------------------------------------------------------ statistics

struct StatsParams {
    LogitsIn in;
    const float *row_w;  // a row with weight 0 is ignored (may be null)
    const int32_t *off;  // rows before off[0] and from off[last] on are ignored (may be null)
    int last;
    float *logp, *lse, *entropy;
    float2 *ms;          // (m, s) of each row (s = 0: nothing to differentiate), may be null
    bool nan_target;     // a target past the vocabulary gives NaN (else it is ignored)
};

template <int DT, bool ENT>
__global__ void __launch_bounds__(THREADS) stats_kernel(const StatsParams P) {
    pdl_wait();
    pdl_trigger();
    const long long row = blockIdx.x;
    const long long tgt = target_of(P.in, row);
    const bool bad = tgt >= P.in.vocab;
    if (tgt < 0 || bad || (P.row_w && P.row_w[row] == 0.f) ||
        (P.off && (row < P.off[0] || row >= P.off[P.last]))) {
        if (threadIdx.x == 0) {
            if (P.logp) P.logp[row] = bad && P.nan_target ? __int_as_float(0x7fffffff) : 0.f;
            if (P.lse) P.lse[row] = 0.f;
            if (P.entropy) P.entropy[row] = 0.f;
            if (P.ms) P.ms[row] = make_float2(0.f, 0.f);
        }
        return;
    }
    const char *z = P.in.logits + row * P.in.ld_bytes;
    const Row<DT> r(z, P.in.vocab);
    const float k = P.in.k;
    Stat<ENT> st;
    const int G = r.groups();
    for (int g = threadIdx.x; g < G; g += THREADS) {
        float v[Elem<DT>::N];
        Elem<DT>::unpack(r.load(g), v);
        st.template add<Elem<DT>::N>(v, k);
    }
    st.merge_lanes(k);
    __shared__ float3 part[THREADS / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = make_float3(st.m, st.s, st.t);
    __syncthreads();
    if (threadIdx.x == 0) {
        Stat<ENT> all;
        for (int i = 0; i < THREADS / 32; ++i) all.merge(part[i].x, part[i].y, part[i].z, k);
        const RowResult q = row_result(all.m, all.s, all.t, logit_at<DT>(z, tgt), P.in.tau);
        if (P.logp) P.logp[row] = q.logp;
        if (P.lse) P.lse[row] = q.lse;
        if (P.entropy) P.entropy[row] = q.h;
        if (P.ms) P.ms[row] = make_float2(all.m, all.s);
    }
}

// ------------------------------------------------------------ gradient

struct GradParams {
    LogitsIn in;
    const float2 *ms;       // (m, s) of each row
    const float *entropy;   // with gh
    const float *g, *gh;    // gradients of logp and H (gh may be null)
    float scale;            // the call's scale / tau
    char *out;
    long long ld_out_bytes;
};

template <int DT, bool ENT>
__global__ void __launch_bounds__(THREADS) grad_kernel(const GradParams P) {
    using E = Elem<DT>;
    pdl_wait();
    pdl_trigger();
    const long long row = blockIdx.x;
    const long long tgt = target_of(P.in, row);
    const Row<DT> r(P.in.logits + row * P.in.ld_bytes, P.in.vocab);
    char *out = P.out + row * P.ld_out_bytes;
    const bool same = (((uintptr_t)out ^ (uintptr_t)(P.in.logits + row * P.in.ld_bytes)) & 15) == 0;
    const float k = P.in.k;
    float g = P.g[row] * P.scale, gh = ENT ? P.gh[row] * P.scale : 0.f;
    const float m = P.ms[row].x, s = P.ms[row].y;
    const int G = r.groups();
    if (tgt < 0 || tgt >= P.in.vocab || s == 0.f || (g == 0.f && gh == 0.f)) {
        float v[E::N];
#pragma unroll
        for (int i = 0; i < E::N; ++i) v[i] = 0.f;
        for (int q = threadIdx.x; q < G; q += THREADS) store_group<DT>(r, q, out, same, v);
        return;
    }
    const float inv = 1.f / s;
    const float b = ENT ? -gh * LN2 * inv : 0.f;
    const float a = ENT ? -(g + gh * (P.entropy[row] - LN2 * log2f(s))) * inv : -g * inv;
    for (int q = threadIdx.x; q < G; q += THREADS) {
        float v[E::N];
        E::unpack(r.load(q), v);
        const int e0 = r.first(q);
#pragma unroll
        for (int i = 0; i < E::N; ++i) {
            const float y = (v[i] - m) * k, e = ex2(y);
            v[i] = ENT ? e * fmaf(b, fmaxf(y, Y_FLOOR), a) : e * a;
            if (e0 + i == tgt) v[i] += g;
        }
        store_group<DT>(r, q, out, same, v);
    }
}

// ------------------------------------------------------------ small kernels

// Index of the last of offsets[0 .. n - 1] (clamped to 0 .. rows) that is <= row, or -1.
__device__ __forceinline__ int sequence_of(const int32_t *off, int n, long long row) {
    int lo = -1, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= row) lo = mid; else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ long long clamp_row(int32_t v, long long rows) {
    return v < 0 ? 0 : v > rows ? rows : v;
}

template <class T>
__device__ __forceinline__ T block_sum(T v, T *part) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    T all = 0;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) all += part[i];
    return all;
}

struct PolicyRows {
    const void *target;
    int target_i32, vocab;
    long long rows;
    const float *weight;
    const float *advantage;
    const int32_t *off;
    int seqs, seq_mean;
    float *row_w, *row_a;  // weight (0: ignored) and advantage of every row
    int *err;
};

// One CTA: each row's weight and advantage.
__global__ void __launch_bounds__(1024) policy_rows_kernel(const PolicyRows P) {
    pdl_wait();
    pdl_trigger();
    __shared__ int part[32];
    auto target = [&](long long row) {
        return P.target_i32 ? (long long)((const int32_t *)P.target)[row] : (long long)((const int64_t *)P.target)[row];
    };
    int n = 0, bad = 0;
    const int ends = P.seqs + 1;
    for (long long row = threadIdx.x; row < P.rows; row += blockDim.x) {
        const long long t = target(row);
        bad |= t >= P.vocab;
        int seq = 0;
        if (P.off) seq = sequence_of(P.off, ends, row);
        const bool in = t >= 0 && t < P.vocab && seq >= 0 && (!P.off || seq < P.seqs);
        n += in;
        P.row_w[row] = in ? (P.weight ? P.weight[row] : 1.f) : 0.f;
        P.row_a[row] = in ? P.advantage[P.off ? seq : row] : 0.f;
    }
    bad = block_sum(bad, part);
    if (threadIdx.x == 0) *P.err = bad ? ERR_TARGET : 0;
    n = block_sum(n, part);
    if (P.weight) return;
    if (!P.seq_mean) {
        for (long long row = threadIdx.x; row < P.rows; row += blockDim.x)
            if (P.row_w[row] != 0.f) P.row_w[row] = 1.f / (float)n;
        return;
    }
    __syncthreads();
    for (int q = threadIdx.x / 32; q < P.seqs; q += blockDim.x / 32) {
        const long long r0 = clamp_row(P.off[q], P.rows), r1 = clamp_row(P.off[q + 1], P.rows);
        int c = 0;
        for (long long row = r0 + (threadIdx.x & 31); row < r1; row += 32) c += P.row_w[row] != 0.f;
        c = __reduce_add_sync(0xffffffffu, c);
        __syncwarp();
        for (long long row = r0 + (threadIdx.x & 31); row < r1; row += 32)
            if (P.row_w[row] != 0.f) P.row_w[row] = 1.f / ((float)P.seqs * (float)c);
    }
}

struct PolicyTerms {
    long long rows;
    const float *row_w, *row_a, *old_logp, *ref_logp;
    const float *logp, *entropy;
    const float2 *ms;
    float clip_low, clip_high, kl_coef, entropy_coef;
    float *kl;            // user's, may be null
    float *g, *gh;        // gradients of logp and H (gh may be null)
    float *stats;
    int *err;
};

// One CTA: the loss terms of every row, their sums and the gradients.
__global__ void __launch_bounds__(1024) policy_terms_kernel(const PolicyTerms P) {
    pdl_wait();
    pdl_trigger();
    __shared__ double part[32];
    double sum[5] = {0, 0, 0, 0, 0};
    int bad = 0;
    for (long long row = threadIdx.x; row < P.rows; row += blockDim.x) {
        const float w = P.row_w[row];
        float g = 0.f, gh = 0.f, kl = 0.f;
        if (w != 0.f) {
            if (P.ms[row].y == 0.f) {
                bad = 1;
            } else {
                const float lp = P.logp[row], a = P.row_a[row], h = P.entropy ? P.entropy[row] : 0.f;
                const float r = expf(lp - P.old_logp[row]);
                const float c = fminf(fmaxf(r, 1.f - P.clip_low), 1.f + P.clip_high);
                const float u = r * a, v = c * a;
                const bool open = !(u > v);
                const float pg = open ? -u : -v;
                float dlp = open ? -u : 0.f;
                if (P.ref_logp) {
                    const float d = P.ref_logp[row] - lp, e = expf(d);
                    kl = e - d - 1.f;
                    dlp += P.kl_coef * (1.f - e);
                }
                const float l = pg + P.kl_coef * kl - P.entropy_coef * h;
                sum[0] += (double)w * l;
                sum[1] += (double)w * pg;
                sum[2] += (double)w * kl;
                sum[3] += (double)w * h;
                sum[4] += open ? 0. : (double)w;
                g = w * dlp;
                gh = -w * P.entropy_coef;
                bad |= !finite(lp) || !finite(l) || !finite(g);
            }
        }
        P.g[row] = g;
        if (P.gh) P.gh[row] = gh;
        if (P.kl) P.kl[row] = kl;
    }
    for (int i = 0; i < 5; ++i) {
        const double s = block_sum(sum[i], part);
        if (threadIdx.x == 0) P.stats[i] = (float)s;
        if (i == 0) bad |= !finite((float)s);
    }
    __shared__ int ipart[32];
    bad = block_sum(bad, ipart);
    if (threadIdx.x == 0 && bad) *P.err |= ERR_NONFINITE;
}

struct PrefPairs {
    const void *target;
    int target_i32, vocab;
    long long rows;
    const int32_t *off;
    int pairs;
    const float *ref, *pair_weight;
    int kind, average;
    float beta, smooth;
    const float *logp;   // of every row (0 where ignored)
    const float2 *ms;
    float *row_g;        // gradient of every row's logp
    double *terms;       // [pairs] weighted f
    int *bad;            // [pairs] error bits
    float *pair_loss, *seq_logp;
};

// ln(1 + e^-x) = -ln sigma(x) without overflow.
__device__ __forceinline__ double softplus_neg(double x) {
    return (x < 0 ? -x : 0.) + log1p(exp(-fabs(x)));
}

// One CTA per pair: the sums of its two sequences, f and its derivative.
__global__ void __launch_bounds__(256) pref_pairs_kernel(const PrefPairs P) {
    pdl_wait();
    pdl_trigger();
    __shared__ double part[8];
    __shared__ int ipart[8];
    const int b = blockIdx.x;
    double l[2];
    int n[2], bad = 0;
    for (int q = 0; q < 2; ++q) {
        const long long r0 = clamp_row(P.off[2 * b + q], P.rows), r1 = clamp_row(P.off[2 * b + q + 1], P.rows);
        double s = 0;
        int c = 0;
        for (long long row = r0 + threadIdx.x; row < r1; row += blockDim.x) {
            const long long t = P.target_i32 ? (long long)((const int32_t *)P.target)[row]
                                             : (long long)((const int64_t *)P.target)[row];
            if (t >= P.vocab) bad |= ERR_TARGET;
            if (t < 0 || t >= P.vocab) continue;
            ++c;
            if (P.ms[row].y == 0.f) {  // every logit -inf: left out
                bad |= ERR_NONFINITE;
                continue;
            }
            if (!finite(P.logp[row])) bad |= ERR_NONFINITE;
            s += P.logp[row];
        }
        s = block_sum(s, part);
        n[q] = block_sum(c, ipart);
        l[q] = P.average && n[q] > 0 ? s / n[q] : s;
        if (!finite((float)l[q])) bad |= ERR_NONFINITE;
        if (threadIdx.x == 0 && P.seq_logp) P.seq_logp[2 * b + q] = (float)l[q];
    }
    const double h = (l[0] - (P.ref ? P.ref[2 * b] : 0.f)) - (l[1] - (P.ref ? P.ref[2 * b + 1] : 0.f));
    const double beta = P.beta, e = P.smooth, x = beta * h;
    double f, d;
    if (P.kind == KFAC_PREF_SIGMOID) {
        f = (1 - e) * softplus_neg(x) + (e > 0 ? e * softplus_neg(-x) : 0.);
        d = beta * (e / (1 + exp(-x)) - (1 - e) / (1 + exp(x)));
    } else if (P.kind == KFAC_PREF_HINGE) {
        f = x < 1 ? 1 - x : x >= 1 ? 0. : x;  // (NaN stays)
        d = x < 1 ? -beta : x >= 1 ? 0. : x;
    } else {
        const double o = h - 0.5 / beta;
        f = o * o;
        d = 2 * o;
    }
    const double v = P.pair_weight ? (double)P.pair_weight[b] : 1.0 / P.pairs;
    if (!finite((float)f)) bad |= ERR_NONFINITE;
    bad = __syncthreads_or(bad & ERR_NONFINITE ? 1 : 0) * ERR_NONFINITE | __syncthreads_or(bad & ERR_TARGET ? 1 : 0) * ERR_TARGET;
    if (threadIdx.x == 0) {
        P.terms[b] = v == 0. ? 0. : v * f;
        P.bad[b] = bad;
        if (P.pair_loss) P.pair_loss[b] = (float)f;
    }
    for (int q = 0; q < 2; ++q) {
        const long long r0 = clamp_row(P.off[2 * b + q], P.rows), r1 = clamp_row(P.off[2 * b + q + 1], P.rows);
        const double dl = v == 0. ? 0. : v * d * (q ? -1 : 1) / (P.average && n[q] > 0 ? n[q] : 1);
        for (long long row = r0 + threadIdx.x; row < r1; row += blockDim.x) P.row_g[row] = (float)dl;
    }
}

struct PrefSum {
    const double *terms;
    const int *bad;
    int pairs;
    float *loss;
    int *err;
};
__global__ void __launch_bounds__(256) pref_sum_kernel(const PrefSum P) {
    pdl_wait();
    pdl_trigger();
    __shared__ double part[8];
    __shared__ int ipart[8];
    double s = 0;
    int bad = 0;
    for (int b = threadIdx.x; b < P.pairs; b += blockDim.x) {
        s += P.terms[b];
        bad |= P.bad[b];
    }
    s = block_sum(s, part);
    const int nf = block_sum(bad & ERR_NONFINITE ? 1 : 0, ipart), tg = block_sum(bad & ERR_TARGET ? 1 : 0, ipart);
    if (threadIdx.x == 0) {
        *P.loss = (float)s;
        *P.err = (nf || !finite((float)s) ? ERR_NONFINITE : 0) | (tg ? ERR_TARGET : 0);
    }
}

// ------------------------------------------------------------ launches

template <class F>
kfac_status by_type(int dtype, bool ent, F &&f) {
    if (dtype == KFAC_BF16) return ent ? f.template run<KFAC_BF16, true>() : f.template run<KFAC_BF16, false>();
    if (dtype == KFAC_F16) return ent ? f.template run<KFAC_F16, true>() : f.template run<KFAC_F16, false>();
    return ent ? f.template run<KFAC_F32, true>() : f.template run<KFAC_F32, false>();
}

struct RunStats {
    const StatsParams &P;
    long long rows;
    cudaStream_t st;
    template <int DT, bool ENT>
    kfac_status run() {
        KFAC_LAUNCH(KK_LOSS_ROWS, st, (stats_kernel<DT, ENT>), (unsigned)rows, THREADS, 0, P);
        return KFAC_OK;
    }
};
struct RunGrad {
    const GradParams &P;
    long long rows;
    cudaStream_t st;
    template <int DT, bool ENT>
    kfac_status run() {
        KFAC_LAUNCH(KK_LOSS_GRAD, st, (grad_kernel<DT, ENT>), (unsigned)rows, THREADS, 0, P);
        return KFAC_OK;
    }
};

size_t elem_size(int dtype) { return dtype == KFAC_F32 ? 4 : 2; }

// The arguments that every call on logits shares.
kfac_status check_logits(int dtype, const void *logits, long long ld, long long rows, int vocab, const void *target,
                         float tau) {
    if (dtype != KFAC_BF16 && dtype != KFAC_F16 && dtype != KFAC_F32) return KFAC_ERR_INVALID;
    if (rows < 0 || vocab < 1 || ld < vocab || (rows > 0 && (!logits || !target))) return KFAC_ERR_INVALID;
    if ((uintptr_t)logits % elem_size(dtype)) return KFAC_ERR_INVALID;
    if (!(tau > 0.f) || !std::isfinite(tau)) return KFAC_ERR_INVALID;
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
    float *row_w, *row_a, *g, *gh, *logp, *h;
    float2 *ms;
};
PolicyPlan plan_policy(const kfac_policy_desc &d, Arena &ws) {
    PolicyPlan p;
    const size_t n = (size_t)d.rows;
    p.err = ws.take<int>(64);
    p.row_w = ws.take<float>(n);
    p.row_a = ws.take<float>(n);
    p.g = ws.take<float>(n);
    p.gh = ws.take<float>(n);
    p.logp = ws.take<float>(n);
    p.h = ws.take<float>(n);
    p.ms = ws.take<float2>(n);
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
    float *logp, *row_g;
    float2 *ms;
    double *terms;
};
PrefPlan plan_preference(const kfac_preference_desc &d, Arena &ws) {
    PrefPlan p;
    const size_t n = (size_t)d.rows;
    p.err = ws.take<int>(64);
    p.logp = ws.take<float>(n);
    p.row_g = ws.take<float>(n);
    p.ms = ws.take<float2>(n);
    p.terms = ws.take<double>((size_t)d.pairs);
    p.bad = ws.take<int>((size_t)d.pairs);
    return p;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" kfac_status kfac_token_logprob(const kfac_logprob_desc *desc, void *stream) {
    if (!desc) return KFAC_ERR_INVALID;
    const kfac_logprob_desc &d = *desc;
    kfac_status s = check_logits(d.dtype, d.logits, d.ld, d.rows, d.vocab, d.target, d.temperature);
    if (s != KFAC_OK) return s;
    if (d.rows == 0) return KFAC_OK;
    if (!d.logp || (uintptr_t)d.saved % 8) return KFAC_ERR_INVALID;
    if (!all_on_this_device({d.logits, d.target, d.logp, d.lse, d.entropy, d.saved})) return KFAC_ERR_INVALID;
    StatsParams P{logits_in(d), nullptr, nullptr, 0, d.logp, d.lse, d.entropy, (float2 *)d.saved, true};
    return by_type(d.dtype, d.entropy != nullptr, RunStats{P, d.rows, (cudaStream_t)stream});
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
    GradParams P{logits_in(d), (const float2 *)d.saved, d.entropy, d.dlogp, d.dentropy, 1.f / d.temperature,
                 (char *)d.dlogits, d.ld_d * (long long)elem_size(d.dtype)};
    return by_type(d.dtype, d.dentropy != nullptr, RunGrad{P, d.rows, (cudaStream_t)stream});
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
    const bool ent = d.entropy_coef != 0.f || d.entropy;
    float *h = d.entropy ? d.entropy : p.h, *logp = d.logp ? d.logp : p.logp;
    PolicyRows R{d.target, d.target_i32, d.vocab, d.rows, d.weight, d.advantage, d.seq_offsets, d.seqs, d.seq_mean,
                 p.row_w, p.row_a, p.err};
    KFAC_LAUNCH(KK_LOSS_SMALL, st, policy_rows_kernel, 1, 1024, 0, R);
    if (d.rows > 0) {
        StatsParams S{logits_in(d), p.row_w, nullptr, 0, logp, nullptr, ent ? h : nullptr, p.ms, false};
        if ((s = by_type(d.dtype, ent, RunStats{S, d.rows, st})) != KFAC_OK) return s;
    }
    const bool ent_grad = d.entropy_coef != 0.f;
    PolicyTerms T{d.rows, p.row_w, p.row_a, d.old_logp, d.ref_logp, logp, ent ? h : nullptr, p.ms, d.clip_low,
                  d.clip_high, d.kl_coef, d.entropy_coef, d.kl, p.g, ent_grad ? p.gh : nullptr, d.stats, p.err};
    KFAC_LAUNCH(KK_LOSS_SMALL, st, policy_terms_kernel, 1, 1024, 0, T);
    if (!d.dlogits || d.rows == 0) return KFAC_OK;
    GradParams G{logits_in(d), p.ms, h, p.g, ent_grad ? p.gh : nullptr, d.grad_scale / d.temperature,
                 (char *)d.dlogits, d.ld_d * (long long)elem_size(d.dtype)};
    return by_type(d.dtype, ent_grad, RunGrad{G, d.rows, st});
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
    KFAC_CUDA_TRY(cudaMemsetAsync(p.row_g, 0, (size_t)d.rows * sizeof(float), st));  // rows of no sequence
    if (d.rows > 0) {
        StatsParams S{logits_in(d), nullptr, d.seq_offsets, 2 * d.pairs, logp, nullptr, nullptr, p.ms, false};
        if ((s = by_type(d.dtype, false, RunStats{S, d.rows, st})) != KFAC_OK) return s;
    }
    PrefPairs Q{d.target, d.target_i32, d.vocab, d.rows, d.seq_offsets, d.pairs, d.ref_logp, d.pair_weight, d.kind,
                d.average, d.beta, d.label_smoothing, logp, p.ms, p.row_g, p.terms, p.bad, d.pair_loss, d.seq_logp};
    KFAC_LAUNCH(KK_LOSS_SMALL, st, pref_pairs_kernel, (unsigned)d.pairs, 256, 0, Q);
    PrefSum U{p.terms, p.bad, d.pairs, d.loss, p.err};
    KFAC_LAUNCH(KK_LOSS_SMALL, st, pref_sum_kernel, 1, 256, 0, U);
    if (!d.dlogits || d.rows == 0) return KFAC_OK;
    GradParams G{logits_in(d), p.ms, nullptr, p.row_g, nullptr, d.grad_scale / d.temperature,
                 (char *)d.dlogits, d.ld_d * (long long)elem_size(d.dtype)};
    return by_type(d.dtype, false, RunGrad{G, d.rows, st});
}
