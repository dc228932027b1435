// loss.cuh -- kernels of the losses on logits: token log-probabilities and their
// gradient, the clipped policy loss with a KL term, and the preference loss over
// pairs.
//
// With y_j = (z_j - m) k, k = log2(e) / tau and m the row's maximum,
//   s = sum_j 2^y_j,  t = sum_j 2^y_j y_j,
//   logp = (z_target - m) / tau - ln s,   lse = m / tau + ln s,
//   H = ln 2 (log2 s - t / s),
// and the gradient of g logp + gh H (times the call's scale, over tau) is
//   d_j = 2^y_j (a + b y_j) + g [j = target],
//   b = - gh ln 2 / s,   a = - (g + gh (H - ln 2 log2 s)) / s.
//
// All of it is bound by memory (a row is read once, its gradient written once; one
// or two powers of two and some ten instructions an element), and by the fixed work
// of a row where rows are short.  Which kernel takes a call, by the whole 16-byte
// groups of a row (RunRows; both sides of each bound were measured):
//   few rows of at most 256 groups    *_small_kernel    the whole loss in one launch
//   up to 512 (1024 without gradient) warp_rows_kernel  8 to 32 lanes to a row, two passes
//   with gradient                     ring_rows_kernel  kept in shared memory
//   statistics alone, or rows that    stream_rows_kernel, then grad_kernel
//   no cluster can keep
#pragma once

#include <algorithm>
#include <atomic>
#include <cmath>

#include "logits.cuh"
#include "ring.h"

namespace kfac {
namespace loss {

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
__device__ __forceinline__ RowResult row_result(const Part &p, float z_t, float tau) {
    RowResult r;
    if (p.s == 0.f) {
        r.logp = r.lse = -INFINITY;
        r.h = 0.f;
        return r;
    }
    const float l2 = log2f(p.s);
    r.logp = (z_t - p.m) / tau - LN2 * l2;
    r.lse = p.m / tau + LN2 * l2;
    r.h = LN2 * (l2 - p.t / p.s);
    return r;
}

// What a row's gradient needs: d_j = 2^y_j (a + b y_j) + g [j = target]; none: zeros.
struct Coef {
    float m, a, b, g;
    bool none;
};
// From the gradients g of logp and gh of H, times the call's scale over tau.
template <bool ENT>
__device__ __forceinline__ Coef coef_of(float m, float s, float h, float g, float gh) {
    Coef c;
    const float inv = 1.f / s;
    c.m = m;
    c.g = g;
    c.b = ENT ? -gh * LN2 * inv : 0.f;
    c.a = ENT ? -(g + gh * (h - LN2 * log2f(s))) * inv : -g * inv;
    c.none = s == 0.f || (g == 0.f && gh == 0.f);
    return c;
}
// The gradient of a group of logits, without the target's g.
template <int DT, bool ENT, bool FAST>
__device__ __forceinline__ uint4 grad_group(uint4 u, const Coef &c, const Shift &h) {
    constexpr int H = Elem<DT>::N / 2;
    f2 v[H];
    unpack_pairs<DT>(ENT && FAST ? Elem<DT>::bounded(u) : u, v);
    const f2 a = pair(c.a, c.a), b = pair(c.b, c.b);
    float f[Elem<DT>::N];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        const f2 y = h.apply<FAST>(v[i]), e = ex2(y);
        const float2 d = both(ENT ? mul(e, fma(b, FAST ? y : max2(y, Y_FLOOR), a)) : mul(e, a));
        f[2 * i] = d.x;
        f[2 * i + 1] = d.y;
    }
    return Elem<DT>::pack(f);
}
// The coefficients for exponents that are delta too large.
__device__ __forceinline__ Coef shifted(Coef c, const Shift &h) {
    const float f = ex2(-h.delta);
    c.a = f * fmaf(-c.b, h.delta, c.a);
    c.b *= f;
    return c;
}
template <bool ENT>
__device__ __forceinline__ float grad_target(float z_t, const Coef &c, float k) {
    const float y = (z_t - c.m) * k;
    return ex2(y) * (ENT ? fmaf(c.b, fmaxf(y, Y_FLOOR), c.a) : c.a) + c.g;
}

// Zeros to n elements that start anywhere, by threads tid of nt.
template <int DT>
__device__ __forceinline__ void zero_row(char *out, int n, int tid, int nt) {
    const Row<DT> o(out, n);
    for (int g = o.begin() + tid; g < o.end(); g += nt)
        *reinterpret_cast<uint4 *>(const_cast<char *>(o.base) + (size_t)g * 16) = make_uint4(0, 0, 0, 0);
    typename Elem<DT>::bits *e = (typename Elem<DT>::bits *)out;
    const int front = min(n, o.first(o.begin())), back = max(front, o.first(o.end()));
    for (int i = tid; i < front; i += nt) e[i] = 0;
    for (int i = back + tid; i < n; i += nt) e[i] = 0;
}
// The gradient of a whole row, read again from its logits, by threads tid of nt.
// Groups lie as the output does; a logits' row that starts elsewhere modulo 16
// bytes is read in shifted pieces.
template <int DT, bool ENT, bool FAST, bool ANY>
__device__ __forceinline__ void grad_groups(const char *z, char *out, int n, int tgt, const Coef &c, float d_t,
                                            const Shift &h, int tid, int nt) {
    using bits = typename Elem<DT>::bits;
    constexpr int N = Elem<DT>::N, BATCH = 4;
    const Row<DT> o(out, n);
    const char *src = z - o.phase * (int)sizeof(bits);  // where the row's group 0 would start
    const int off = (int)((uintptr_t)src & 15);
    const int a = ANY ? (N + o.phase + N - 1) / N : o.begin(), b = ANY ? max(a, (n + o.phase) / N - 1) : o.end();
    char *to = const_cast<char *>(o.base);
    for (int g = a + tid; g < b; g += BATCH * nt) {
        Pieces<1, ANY> u[BATCH];
        if (g + (BATCH - 1) * nt < b) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) u[i].load(src + (size_t)(g + i * nt) * 16, off);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                uint4 v;
                u[i].take(off, &v);
                *reinterpret_cast<uint4 *>(to + (size_t)(g + i * nt) * 16) = grad_group<DT, ENT, FAST>(v, c, h);
            }
        } else {
            for (int q = g; q < b; q += nt) {
                uint4 v;
                u[0].load(src + (size_t)q * 16, off);
                u[0].take(off, &v);
                *reinterpret_cast<uint4 *>(to + (size_t)q * 16) = grad_group<DT, ENT, FAST>(v, c, h);
            }
        }
    }
    // the elements before and behind: groups 0 .. a - 1 and b .. , at most two of each
    const int rest = min(a, o.groups()) + max(0, o.groups() - max(a, b));
    for (int i = nt - 1 - tid; i < rest; i += nt) {
        const int g = i < a ? i : max(a, b) + (i - a), e0 = o.first(g);
        Row<DT>::store_edge(out, e0, n, grad_group<DT, ENT, FAST>(Row<DT>::edge_group(z + (long long)e0 * (int)sizeof(bits), e0, n), c, h));
    }
    // the thread that wrote the target's group writes the target's own value
    const int tg = (tgt + o.phase) / N;
    const int owner = tg >= a && tg < b ? (tg - a) % nt : nt - 1 - (tg < a ? tg : a + tg - max(a, b)) % nt;
    if (tid == owner) ((bits *)out)[tgt] = Elem<DT>::round(d_t);
}
template <int DT, bool ENT>
__device__ __noinline__ void grad_groups_any(const char *z, char *out, int n, int tgt, const Coef &c, float d_t,
                                             const Shift &h, int tid, int nt) {
    grad_groups<DT, ENT, true, true>(z, out, n, tgt, c, d_t, h, tid, nt);
}
template <int DT, bool ENT>
__device__ __noinline__ void grad_groups_slow(const char *z, char *out, int n, int tgt, const Coef &c, float d_t,
                                              const Shift &h, int tid, int nt) {
    grad_groups<DT, ENT, false, true>(z, out, n, tgt, c, d_t, h, tid, nt);
}
template <int DT, bool ENT>
__device__ __forceinline__ void grad_row(const char *z, char *out, int n, int tgt, float z_t, const Coef &c, float k,
                                         int tid, int nt) {
    const Shift h = shift_of<DT, ENT>(c.m, k, c.b);
    const float d_t = grad_target<ENT>(z_t, c, k);
    if (h.ok && (((uintptr_t)out ^ (uintptr_t)z) & 15) == 0)
        grad_groups<DT, ENT, true, false>(z, out, n, tgt, shifted(c, h), d_t, h, tid, nt);
    else if (h.ok)
        grad_groups_any<DT, ENT>(z, out, n, tgt, shifted(c, h), d_t, h, tid, nt);
    else grad_groups_slow<DT, ENT>(z, out, n, tgt, c, d_t, h, tid, nt);
}

template <int DT, bool ENT>
__device__ __noinline__ void grad_row_apart(const char *z, char *out, int n, int tgt, float z_t, const Coef &c, float k,
                                            int tid, int nt) {
    grad_row<DT, ENT>(z, out, n, tgt, z_t, c, k, tid, nt);
}

// ------------------------------------------------------------ rows

// Sum over a block; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int *part) {
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    int all = (int)(threadIdx.x & 31) < (int)blockDim.x / 32 ? part[threadIdx.x & 31] : 0;
    return __reduce_add_sync(0xffffffffu, all);
}
// Sum over a block, in a fixed order; thread 0 gets it.
__device__ __forceinline__ Wide block_sum(Wide v, Wide *part) {
    v.add_lanes();
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    Wide all{};
    if (threadIdx.x < 32) {
        if ((int)threadIdx.x < (int)blockDim.x / 32) all = part[threadIdx.x];
        all.add_lanes();
    }
    return all;
}
// Another CTA's copy of a shared variable.
template <class T>
__device__ __forceinline__ T *peer(T *local, int rank) {
    T *p;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(p) : "l"(local), "r"(rank));
    return p;
}

// A row's terms of the policy loss: w l, w pg, w kl, w H, w [clipped], and whether
// one of its values is not finite.
struct Terms {
    float4 t;
    float2 f;
};
// Sums of rows' terms.
struct TermSums {
    Wide sum[5];
    int bad;
    __device__ __forceinline__ void add(const Terms &o) {
        sum[0].add(o.t.x);
        sum[1].add(o.t.y);
        sum[2].add(o.t.z);
        sum[3].add(o.t.w);
        sum[4].add(o.f.x);
        bad |= o.f.y != 0.f;
    }
    __device__ __forceinline__ void add(const TermSums &o) {
#pragma unroll
        for (int i = 0; i < 5; ++i) sum[i].add(o.sum[i]);
        bad |= o.bad;
    }
    // Over the block, in a fixed order; thread 0's is the one to take.
    __device__ __forceinline__ void add_block() {
        __shared__ Wide part[5][32];
        __shared__ int bad_of[32];
        const int lane = threadIdx.x % 32, w = threadIdx.x / 32, warps = blockDim.x / 32;
        bad = __reduce_or_sync(ALL_LANES, bad);
#pragma unroll
        for (int i = 0; i < 5; ++i) sum[i].add_lanes();
        __syncthreads();
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 5; ++i) part[i][w] = sum[i];
            bad_of[w] = bad;
        }
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            sum[i] = lane < warps ? part[i][lane] : Wide{};
            sum[i].add_lanes();
        }
        bad = __reduce_or_sync(ALL_LANES, lane < warps ? bad_of[lane] : 0);
    }
    __device__ __forceinline__ void write(float *stats, int *err, int word) const {
        float v = 0.f;
#pragma unroll
        for (int i = 4; i >= 0; --i) stats[i] = v = (float)sum[i].value();
        if (bad || !finite(v)) word |= ERR_NONFINITE;
        if (word) atomicOr(err, word);
    }
};

// A row of the policy loss: its target (-1: ignored), weight, advantage and
// log-probability under the policy that drew it.
struct __align__(16) PolicyRow {
    int target;
    float weight, advantage, old_logp;
};

struct RowParams {
    LogitsIn in;
    long long rows;
    const int32_t *off;        // rows before off[0] and from off[last] on are ignored (may be null)
    int last;
    bool nan_target;           // a target past the vocabulary gives NaN (else it is ignored)
    float *logp, *lse, *entropy;
    float2 *ms;                // (m, s) of each row (s = 0: nothing to differentiate), may be null
    // policy loss
    bool policy;               // the policy loss, its rows' other inputs in meta
    const PolicyRow *meta;
    const int *order;          // the order in which the ring takes the rows (live ones first)
    const float *ref_logp;
    float clip_low, clip_high, kl_coef, entropy_coef;
    float *kl;
    TermSums *sums;            // one for each CTA (or cluster) of the launch, the last of which adds them up
    unsigned *done;            // ... counted here (0 before the launch)
    float *stats;
    float2 *g;                 // gradients of logp and H, where the logits' gradient comes later (may be null)
    int *err;
    unsigned *zero;            // a counter and a vector of the calls after this one: set to 0 here (rows that
    float *zero_g;             // are ignored), both may be null
    float scale;               // the call's scale / tau (1 for a call without gradient)
    char *dlogits;             // may be null
    long long ld_d_bytes;
};

// A row's inputs besides its logits.  target < 0: ignored.
__device__ __forceinline__ PolicyRow row_meta(const RowParams &P, long long row) {
    if (P.meta) return *reinterpret_cast<const PolicyRow *>(P.meta + row);
    const long long t = target_of(P.in, row);
    PolicyRow q{t >= 0 && t < P.in.vocab ? (int)t : -1, 0.f, 0.f, 0.f};
    if (P.off && (row < P.off[0] || row >= P.off[P.last])) q.target = -1;
    return q;
}

// An ignored row's outputs.
__device__ __forceinline__ void ignore_row(const RowParams &P, long long row) {
    if (P.logp)
        P.logp[row] = P.nan_target && target_of(P.in, row) >= P.in.vocab ? __int_as_float(0x7fffffff) : 0.f;
    if (P.lse) P.lse[row] = 0.f;
    if (P.entropy) P.entropy[row] = 0.f;
    if (P.ms) P.ms[row] = make_float2(0.f, 0.f);
    if (P.kl) P.kl[row] = 0.f;
    if (P.g) P.g[row] = make_float2(0.f, 0.f);
    if (P.zero_g) P.zero_g[row] = 0.f;
}

// e^d - 1 - d from d and em = e^d - 1.  Near 0 the difference is d^2 / 2 and would be lost
// beside d: up to 1/4 it is d^2 times the series of its quotient, whose first term left
// out is 1.2e-8 of it at 1/4.
__device__ __forceinline__ float kl_term(float d, float em) {
    if (!(fabsf(d) < 0.25f)) return em - d;
    const float q = fmaf(fmaf(fmaf(fmaf(fmaf(1.f / 5040, d, 1.f / 720), d, 1.f / 120), d, 1.f / 24), d, 1.f / 6), d, 0.5f);
    return d * d * q;
}

// A row's outputs (where `write`), its terms and the coefficients of its gradient.
template <bool ENT>
__device__ __forceinline__ Coef finish_row(const RowParams &P, long long row, const PolicyRow &q, float ref,
                                           const Part &p, float z_t, bool write, Terms &o) {
    const RowResult r = row_result(p, z_t, P.in.tau);
    if (write) {
        if (P.logp) P.logp[row] = r.logp;
        if (P.lse) P.lse[row] = r.lse;
        if (P.entropy) P.entropy[row] = r.h;
        if (P.ms) P.ms[row] = make_float2(p.m, p.s);
    }
    if (!P.policy) return Coef{};
    float g = 0.f, gh = 0.f, kl = 0.f, clipped = 0.f, bad = 1.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.s != 0.f) {
        const float w = q.weight, ratio = expf(r.logp - q.old_logp);
        const float c = fminf(fmaxf(ratio, 1.f - P.clip_low), 1.f + P.clip_high);
        const float u = ratio * q.advantage, v = c * q.advantage;
        const bool open = !(u > v);
        const float pg = open ? -u : -v;
        float dlp = open ? -u : 0.f;
        if (P.ref_logp) {
            const float d = ref - r.logp, em = expm1f(d);
            kl = kl_term(d, em);
            dlp -= P.kl_coef * em;
        }
        const float h = ENT ? r.h : 0.f, l = pg + P.kl_coef * kl - P.entropy_coef * h;
        t = make_float4(w * l, w * pg, w * kl, w * h);
        clipped = open ? 0.f : w;
        g = w * dlp;
        gh = -w * P.entropy_coef;
        bad = finite(r.logp) && finite(t.x) && finite(g * P.scale) && (!ENT || finite(gh * P.scale)) ? 0.f : 1.f;
    }
    o.t = t;
    o.f = make_float2(clipped, bad);
    if (write) {
        if (P.kl) P.kl[row] = kl;
        if (P.g) P.g[row] = make_float2(g, gh);
    }
    return coef_of<ENT>(p.m, p.s, r.h, g * P.scale, gh * P.scale);
}

// The groups of a row that a thread keeps in registers between the row's
// statistics and its gradient: group first + i step for i < count (at most VPT),
// below `end`, and perhaps one of the row's edges.
template <int DT, int VPT>
struct Kept {
    uint4 u[VPT];
    int g0, step, end, at;
    // `most`: how many groups any thread of the row has at most.  A thread without
    // the last one loads the row's last whole group in its place.
    __device__ __forceinline__ void load(const Row<DT> &r, int g0_, int step_, int end_, int most, int at_) {
        g0 = g0_;
        step = step_;
        end = end_;
        at = at_;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < most) u[i] = r.load_whole(min(g0 + i * step, end - 1));
    }
    __device__ __forceinline__ float largest(const Row<DT> &r, int most) const {
        auto m = Elem<DT>::lowest();
        if (at >= 0) m = Elem<DT>::raise(m, r.load_edge(at));
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < most) m = Elem<DT>::raise(m, u[i]);
        return Elem<DT>::largest(m);
    }
    template <bool ENT>
    __device__ __forceinline__ Sums<DT, ENT> sums(const Row<DT> &r, const Shift &h, int most, bool edges) const {
        Sums<DT, ENT> s;
        if (h.ok) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (i < most && g0 + i * step < end) s.template add<true>(u[i], h);
        } else {
            for (int g = g0; g < end; g += step) s.template add<false>(r.load_whole(g), h);
        }
        if (edges) {
            const uint4 u = at >= 0 ? r.load_edge(at) : Row<DT>::none();
            if (h.ok) s.template add<true>(u, h);
            else s.template add<false>(u, h);
        }
        return s;
    }
    // The gradient of its groups; `out` starts as the row does modulo 16 bytes.
    template <bool ENT>
    __device__ __forceinline__ void gradient(const Row<DT> &r, char *out, const Coef &c, const Shift &h, int most) const {
        char *o = out - r.phase * sizeof(typename Row<DT>::bits);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < most && g0 + i * step < end)
                *reinterpret_cast<uint4 *>(o + (size_t)(g0 + i * step) * 16) = grad_group<DT, ENT, true>(u[i], c, h);
        if (at >= 0) Row<DT>::store_edge(out, r.first(at), r.n, grad_group<DT, ENT, true>(r.load_edge(at), c, h));
    }
    // Whether this thread writes the target's element.
    __device__ __forceinline__ bool owns(const Row<DT> &r, int target) const {
        const int g = (target + r.phase) / Elem<DT>::N;
        return g == at || (g >= g0 && g < end && (g - g0) % step == 0);
    }
};

// The gradient of a row whose thread's share is in `kept`.
template <int DT, bool ENT, int VPT>
__device__ __forceinline__ void write_gradient(const Kept<DT, VPT> &kept, const Row<DT> &r, const char *z, char *out,
                                               int target, float z_t, const Coef &c, float k, int most, int tid, int nt) {
    if (c.none) {
        zero_row<DT>(out, r.n, tid, nt);
        return;
    }
    const Shift h = shift_of<DT, ENT>(c.m, k, c.b);
    if (!h.ok || (((uintptr_t)out ^ (uintptr_t)z) & 15) != 0) {
        grad_row<DT, ENT>(z, out, r.n, target, z_t, c, k, tid, nt);
        return;
    }
    kept.template gradient<ENT>(r, out, shifted(c, h), h, most);
    // the thread that wrote the target's group adds its g
    if (kept.owns(r, target))
        ((typename Row<DT>::bits *)out)[target] = Elem<DT>::round(grad_target<ENT>(z_t, c, k));
}

// The end of a launch over rows of the policy loss: CTA (or cluster) i of n leaves its
// sums, the last to come adds up all of them, in their order.  Every thread of the
// block comes here; thread 0 holds the block's sums.
__device__ __forceinline__ void leave_sums(const RowParams &P, const TermSums &mine, int i, int n) {
    __shared__ bool last;
    if (threadIdx.x == 0) {
        P.sums[i] = mine;
        __threadfence();
        last = atomicAdd(P.done, 1u) == (unsigned)n - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    TermSums all{};
    for (int c = threadIdx.x; c < n; c += blockDim.x) all.add(P.sums[c]);
    all.add_block();
    if (threadIdx.x == 0) all.write(P.stats, P.err, 0);
}

// One row to L lanes of a warp (L = 8 or 32): rows of at most NV L whole groups.
// All lanes of a warp come here together (the reductions name them all); `in`:
// there is such a row.  (For many rows the two passes of warp_rows_kernel are faster:
// 60000 x 500 bf16 took 84 us by eight lanes of these and takes 72.)
constexpr int NV = 8;
template <int DT, bool ENT, int L>
__device__ __forceinline__ Terms lane_row(const RowParams &P, long long row, bool in, const PolicyRow &q) {
    const int lane = threadIdx.x % L;
    const bool live = q.target >= 0;
    const char *z = P.in.logits + (in ? row : 0) * P.in.ld_bytes;
    const Row<DT> r(z, P.in.vocab);
    const int most = live ? (r.end() - r.begin() + L - 1) / L : 0;
    Kept<DT, NV> kept;
    kept.load(r, r.begin() + lane, L, live ? r.end() : 0, most,
              !live ? -1 : lane == 0 && r.has_front() ? 0 : lane == 1 && r.has_back() ? r.end() : -1);
    const float z_t = live ? logit_at<DT>(z, q.target) : 0.f, ref = live && P.ref_logp ? P.ref_logp[row] : 0.f;
    const Shift h = shift_of<DT, ENT>(lanes_max(kept.largest(r, most), L), P.in.k);
    const Part p = kept.template sums<ENT>(r, h, most, true).part(h, L);
    char *out = P.dlogits ? P.dlogits + (in ? row : 0) * P.ld_d_bytes : nullptr;
    Terms terms{};
    if (!live) {
        if (in && lane == 0) ignore_row(P, row);
        if (in && out) zero_row<DT>(out, P.in.vocab, lane, L);
        return terms;
    }
    const Coef c = finish_row<ENT>(P, row, q, ref, p, z_t, lane == 0, terms);
    if (out) write_gradient<DT, ENT>(kept, r, z, out, q.target, z_t, c, P.in.k, most, lane, L);
    return terms;
}

constexpr int MAX_CLUSTER = 8;
// Stores a part into CTA `rank`'s copy of a shared variable.
__device__ __forceinline__ void store_part(const float4 *local, int rank, float4 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// Rows of middling length, each to L lanes of a warp (L = 8, 16 or 32, for at most 32 L
// whole groups): a first pass for the statistics, a second for the gradient, which
// finds the row in the L2 cache (the rows in flight hold at most 80 MB).  No
// barriers, and the next row's inputs are asked for before a row is begun.  Fewer
// lanes share a row's fixed work, about 600 instructions, among more rows.  A call for
// the log-probabilities of 16000 x 2100 bf16 (67 MB) takes 22 us (26 by 32 lanes always,
// 55 by a CTA to a row), the policy loss of 16000 x 2040 57 us (131 MB) and of 8000 x 4096
// 47: bound by the latency of the two passes over a row and of their reductions.  CTAs of
// 128 threads take the same, of 64 threads 6 to 10 us more with the gradient.
constexpr int WARP_GROUPS = 1024, WARP_GRAD_GROUPS = 512, WARP_SHORT = 64, WARP_THREADS = 256, WARP_PER_SM = 4;
template <int DT, bool ENT, int L>
__global__ void __launch_bounds__(WARP_THREADS, WARP_PER_SM) warp_rows_kernel(const __grid_constant__ RowParams P) {
    constexpr int G = WARP_THREADS / L, BATCH = 4;
    __shared__ TermSums group_sums[G];  // (registers are short)
    pdl_wait();
    pdl_trigger();
    if (P.zero && blockIdx.x == 0 && threadIdx.x == 0) *P.zero = 0;
    const int lane = threadIdx.x % L;
    const unsigned mask = L == 32 ? ALL_LANES : ((1u << L) - 1) << (threadIdx.x % 32 / L * L);
    const float k = P.in.k;
    const long long step = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + threadIdx.x / L;
    TermSums &mine = group_sums[threadIdx.x / L];
    if (lane == 0) mine = TermSums{};
    PolicyRow q{-1, 0.f, 0.f, 0.f};
    if (row < P.rows) q = row_meta(P, row);
    for (; row < P.rows; row += step) {
        const PolicyRow now = q;
        if (row + step < P.rows) q = row_meta(P, row + step);
        char *out = P.dlogits ? P.dlogits + row * P.ld_d_bytes : nullptr;
        if (now.target < 0) {
            if (lane == 0) ignore_row(P, row);
            if (out) zero_row<DT>(out, P.in.vocab, lane, L);
            continue;
        }
        const char *z = P.in.logits + row * P.in.ld_bytes;
        const Row<DT> r(z, P.in.vocab);
        const float z_t = logit_at<DT>(z, now.target), ref = P.ref_logp ? P.ref_logp[row] : 0.f;
        Running<DT, ENT> run(k);
        const int end = r.end();
        int g = r.begin() + lane;
        for (; g - lane + BATCH * L <= end; g += BATCH * L) {
            uint4 u[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) u[i] = r.load_whole(g + i * L);
            run.template add<BATCH>(u, BATCH, 0);
        }
        if (g - lane < end) {
            uint4 u[BATCH];
            const int most = (end - (g - lane) + L - 1) / L;
            unsigned skip = 0;
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i < most) {
                    u[i] = r.load_whole(min(g + i * L, end - 1));
                    skip |= (g + i * L >= end ? 1u : 0u) << i;
                }
            run.template add<BATCH>(u, most, skip);
        }
        const int at = lane == 0 && r.has_front() ? 0 : lane == 1 && r.has_back() ? end : -1;
        if (at >= 0) {
            const uint4 u = r.load_edge(at);
            run.template add<1>(&u, 1, 0);
        }
        __syncwarp(mask);
        const Part p = run.part(L, mask);
        Terms terms{};
        const Coef c = finish_row<ENT>(P, row, now, ref, p, z_t, lane == 0, terms);
        if (P.policy && lane == 0) mine.add(terms);
        if (!out) continue;
        if (c.none) zero_row<DT>(out, P.in.vocab, lane, L);
        else grad_row<DT, ENT>(z, out, P.in.vocab, now.target, z_t, c, k, lane, L);
    }
    if (!P.policy) return;
    __syncthreads();
    TermSums sums = threadIdx.x < G ? group_sums[threadIdx.x] : TermSums{};
    sums.add_block();
    leave_sums(P, sums, blockIdx.x, gridDim.x);
}
// The lanes to a row: as few as its length allows, while they fill the GPU (with 32
// lanes always, log-probabilities of 16000 x 2100 bf16 take 26 us in place of 22).
inline int lanes_of(long long whole, long long rows) {
    int L = 32;
    while (L > 8 && whole <= 16 * L && rows * L > device_sm_count() * 1024LL) L /= 2;
    return L;
}

// The parts of one row from all warps that worked on it, joined by one warp.
template <bool ENT>
__device__ __forceinline__ Part join_parts(const float4 *parts, int n, float k) {
    const int lane = threadIdx.x % 32;
    float M = -F32_MAX;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, parts[i].x);
    M = lanes_max(M, 32);
    Part all{M, 0.f, 0.f};
    for (int i = lane; i < n; i += 32) {
        const float4 v = parts[i];
        const Part p = relative_to<ENT>(Part{v.x, v.y, v.z}, M, k);
        all.s += p.s;
        all.t += p.t;
    }
    all.s = lanes_sum(all.s, 32);
    if (ENT) all.t = lanes_sum(all.t, 32);
    return all;
}

// Statistics only: one row to a CTA or, where there are few rows, to a cluster
// of cs CTAs, each with a run of the row's groups.  Small CTAs, eight to an SM: the
// time between a row's last load and the next one's first is then some other row's
// loading time.  12000 x 128000 bf16 (2.15 GB live) takes 328 us, 6.6 TB/s;
// 4099 x 50001 fp16 (410 MB) 73 us, 5.6 TB/s.  256 threads, six to an SM, take 8% more at
// 6000 x 32000 and the same elsewhere within 3%; four to an SM up to 10% more, batches of two
// groups up to 15% more.  The rows through a shared-memory ring took 104 us in place of 73.
constexpr int STREAM_THREADS = 128, STREAM_PER_SM = 8, BATCH = 4;
template <int DT, bool ENT>
__global__ void __launch_bounds__(STREAM_THREADS, STREAM_PER_SM) stream_rows_kernel(const __grid_constant__ RowParams P, int cs) {
    constexpr int T = STREAM_THREADS, W = T / 32;
    __shared__ float4 parts[2][MAX_CLUSTER * W];
    if (cs > 1) cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, rank = cs > 1 ? blockIdx.x % cs : 0;
    if (P.zero && blockIdx.x == 0 && tid == 0) *P.zero = 0;
    const float k = P.in.k;
    const long long step = gridDim.x / cs;
    int turn = 0;
    __shared__ TermSums sums;  // (registers are short)
    if (tid == 0) sums = TermSums{};
    if (cs > 1) cluster_wait();
    for (long long row = blockIdx.x / cs; row < P.rows; row += step) {
        const PolicyRow q = row_meta(P, row);
        if (q.target < 0) {
            if (rank == 0 && tid == 0) ignore_row(P, row);
            continue;
        }
        const char *z = P.in.logits + row * P.in.ld_bytes;
        const Row<DT> r(z, P.in.vocab);
        const int per = (r.end() - r.begin() + cs - 1) / cs;
        const int c0 = r.begin() + rank * per, g1 = min(r.end(), c0 + per);
        const int at = rank != 0 ? -1 : tid == 0 && r.has_front() ? 0 : tid == 1 && r.has_back() ? r.end() : -1;
        Running<DT, ENT> run(k);
        int g = c0 + tid;
        for (; g - tid + BATCH * T <= g1; g += BATCH * T) {
            uint4 u[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) u[i] = r.load_whole(g + i * T);
            run.template add<BATCH>(u, BATCH, 0);
        }
        if (g - tid < g1) {
            uint4 u[BATCH];
            const int most = (g1 - (g - tid) + T - 1) / T;
            unsigned skip = 0;
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i < most) {
                    u[i] = r.load_whole(min(g + i * T, g1 - 1));
                    skip |= (g + i * T >= g1 ? 1u : 0u) << i;
                }
            run.template add<BATCH>(u, most, skip);
        }
        if (at >= 0) {
            const uint4 u = r.load_edge(at);
            run.template add<1>(&u, 1, 0);
        }
        const Part mine = run.part();
        const float4 packed = make_float4(mine.m, mine.s, mine.t, 0.f);
        if (cs > 1) {
            if (tid % 32 < cs) store_part(&parts[turn][rank * W + tid / 32], tid % 32, packed);
            cluster_sync();
        } else {
            if (tid % 32 == 0) parts[turn][tid / 32] = packed;
            __syncthreads();
        }
        if (tid < 32) {
            // (both are in the L2 cache or on their way to it)
            const float z_t = logit_at<DT>(z, q.target), ref = P.ref_logp ? P.ref_logp[row] : 0.f;
            const Part all = join_parts<ENT>(parts[turn], cs * W, k);
            Terms terms{};
            finish_row<ENT>(P, row, q, ref, all, z_t, rank == 0 && tid == 0, terms);
            if (P.policy && tid == 0) sums.add(terms);
        }
        turn ^= 1;  // the parts of the row after next come after the next row's barrier
    }
    if (P.policy && rank == 0) leave_sums(P, sums, blockIdx.x / cs, (int)step);
}

// Statistics and gradient of rows that a cluster of cs CTAs keeps in shared
// memory: a persistent CTA on each SM, a warp that fetches the coming rows' runs
// of groups into a ring of stages (one bulk copy each), and two teams of warps
// that take the rows in turn, so that one computes while the other waits for
// its row's statistics to be joined (four or eight teams where runs are short).  A
// team's warps send their parts to every CTA of the cluster, each of which joins them
// itself.  Three short passes over a stage (maximum, sums, gradient) need few registers
// and no rescaling; the logits cross HBM once, the gradient is stored as it is made.
// 16391 x 131072 bf16 (8.16 GB) takes 1208 us, 6.8 TB/s, as fast as a copy; a call on
// 2048 x 32768 (242 MB) 51 us, 4.7 TB/s: there the first stages' loading and the last
// ones' storing have nothing beside them.  The row in the registers of a cluster of
// ordinary CTAs took 1770 us, a second pass over the row from memory 1980.
constexpr int TEAM_THREADS = 512, RING_THREADS = TEAM_THREADS + 32, MAX_STAGES = 16;
constexpr int RING_BYTES = 221184;  // of shared memory for the stages: three of 4608 groups

struct __align__(16) StageInputs {
    PolicyRow q;
    int row;
    float ref, z_t;
};
struct StageRow : StageInputs {
    uint4 edge[2];  // the groups before and behind the whole ones (of the cluster's first CTA)
};
template <int TEAMS>
struct RingShared {
    static constexpr int TEAM = TEAM_THREADS / TEAMS, TEAM_WARPS = TEAM / 32;
    float4 parts[TEAMS][2][MAX_CLUSTER * TEAM_WARPS];
    Coef coef[TEAMS][2];
    StageRow row[MAX_STAGES];
    long long given[MAX_STAGES];  // the row (counted within the cluster) that the stage was given to last
    uint64_t full[MAX_STAGES], empty[MAX_STAGES], joined[TEAMS][2];
    TermSums sums[TEAMS];
    int dead;
};

// Asks for bytes (a multiple of 16, on a 16-byte boundary) to come to the L2 cache.
__device__ __forceinline__ void bulk_prefetch(const void *src, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// Stores a part into CTA `rank`'s copy of a shared variable and counts its
// bytes on that CTA's barrier.
__device__ __forceinline__ void send_part(const float4 *local, const uint64_t *bar, int rank, float4 v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
                 : "memory");
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// The team's barrier; whether any of its threads gave true, the same for all of them.
template <int TEAM>
__device__ __forceinline__ bool team_any(int team, bool v) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(team + 1), "r"(TEAM), "r"((uint32_t)v)
        : "memory");
    return any != 0;
}

// A thread's sums over its groups of a stage.
template <int DT, bool ENT, bool FAST, int TEAM>
__device__ __forceinline__ Sums<DT, ENT> stage_sums(const uint4 *stage, int t, int G, const Shift &h) {
    Sums<DT, ENT> s;
#pragma unroll 4
    for (int g = t; g < G; g += TEAM) s.template add<FAST>(stage[g], h);
    return s;
}
template <int DT, bool ENT, int TEAM>
__device__ __noinline__ Sums<DT, ENT> stage_sums_slow(const uint4 *stage, int t, int G, const Shift &h) {
    return stage_sums<DT, ENT, false, TEAM>(stage, t, G, h);
}

// A stage as a thread of a team waits for it (wait_stage).  The row's number is
// released by the thread that has given the stage to it and acquired here, so that
// the barrier's state that is looked at next is no older.
template <class Shared>
struct StageWait {
    Shared &sh;
    int st;
    uint64_t limit_ns = 2000000000ull, t0 = 0;
    __device__ __forceinline__ long long given() const {
        long long n;
        asm volatile("ld.acquire.cta.shared::cta.b64 %0, [%1];" : "=l"(n) : "r"(smem_u32(&sh.given[st])) : "memory");
        return n;
    }
    __device__ __forceinline__ void give(long long n) const {
        asm volatile("st.release.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&sh.given[st])), "l"(n) : "memory");
    }
    __device__ __forceinline__ void start() { t0 = global_timer_ns(); }
    __device__ __forceinline__ bool late() const { return global_timer_ns() - t0 > limit_ns; }
    __device__ __forceinline__ bool wait_full(int parity) const { return mbar_wait(&sh.full[st], parity, limit_ns); }
    __device__ __forceinline__ bool all(bool ok) const { return __all_sync(ALL_LANES, ok); }
    __device__ __forceinline__ StageInputs row() const { return sh.row[st]; }
};

template <int DT, bool ENT, int TEAMS>
__global__ void __launch_bounds__(RING_THREADS, 1) ring_rows_kernel(const __grid_constant__ RowParams P, int cs, int stages,
                                                                    int stage_bytes) {
    constexpr int TEAM = RingShared<TEAMS>::TEAM, TEAM_WARPS = RingShared<TEAMS>::TEAM_WARPS;
    extern __shared__ __align__(128) char ring[];
    __shared__ RingShared<TEAMS> sh;
    const int tid = threadIdx.x, rank = blockIdx.x % cs;
    const float k = P.in.k;
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            sh.given[i] = -1;
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], TEAM_WARPS);
        }
        for (int i = 0; i < 2 * TEAMS; ++i) mbar_init(&sh.joined[i / 2][i % 2], 1);
        sh.dead = 0;
        for (int i = 0; i < TEAMS; ++i) sh.sums[i] = TermSums{};
        fence_barrier_init();
    }
    const long long first = blockIdx.x / cs, step = gridDim.x / cs;
    const long long count = first < P.rows ? (P.rows - first + step - 1) / step : 0;  // rows of this cluster
    // a CTA's run of a row's whole groups
    auto run_of = [&](const Row<DT> &r, int &c0, int &g1) {
        const int per = (r.end() - r.begin() + cs - 1) / cs;
        c0 = r.begin() + rank * per;
        g1 = min(r.end(), c0 + per);
    };
    // While the table of rows is made: as many of the first logits on their way to L2 as the
    // first stages take, whichever rows these will be (2000 x 50001: 94 -> 91 us; two or four
    // rows for one gain less).
    if (tid == TEAM_THREADS && count > 0) {
        const Row<DT> r(P.in.logits + first * P.in.ld_bytes, P.in.vocab);
        int c0, g1;
        run_of(r, c0, g1);
        if (g1 > c0) bulk_prefetch(r.base + (size_t)c0 * 16, (g1 - c0) * 16);
    }
    cluster_sync();
    pdl_wait();
    pdl_trigger();

    if (tid >= TEAM_THREADS) {  // ---- the warp that fetches
        const int lane = tid % 32;
        bool ok = true;
        for (long long n0 = 0; n0 < count && ok; n0 += 32) {
            // the inputs of 32 rows at once, one to a lane
            StageRow mine{};
            mine.q.target = -1;
            if (n0 + lane < count) {
                const long long row = P.order[first + (n0 + lane) * step];
                mine.row = (int)row;
                mine.q = row_meta(P, row);
                if (mine.q.target >= 0) {
                    const char *z = P.in.logits + row * P.in.ld_bytes;
                    mine.z_t = logit_at<DT>(z, mine.q.target);
                    if (rank == 0) {
                        const Row<DT> r(z, P.in.vocab);
                        if (r.has_front()) mine.edge[0] = r.load_edge(0);
                        if (r.has_back()) mine.edge[1] = r.load_edge(r.end());
                    }
                    if (P.ref_logp) mine.ref = P.ref_logp[row];
                }
            }
            for (int j = 0; j < 32 && n0 + j < count; ++j) {
                const long long n = n0 + j;
                const int st = (int)(n % stages);
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[st], (int)(n / stages & 1) ^ 1));
                if (!ok) break;
                if (lane == j) {
                    // (the copy may count its bytes before they are expected: the stage stays open until
                    // this thread has arrived, and then it holds the row's other inputs too)
                    const Row<DT> r(P.in.logits + mine.row * P.in.ld_bytes, P.in.vocab);
                    int c0, g1;
                    run_of(r, c0, g1);
                    const bool loads = mine.q.target >= 0 && g1 > c0;
                    if (loads)
                        bulk_load(ring + (size_t)st * stage_bytes, r.base + (size_t)c0 * 16, (uint32_t)(g1 - c0) * 16,
                                  &sh.full[st]);
                    sh.row[st] = mine;
                    StageWait<RingShared<TEAMS>>{sh, st}.give(n);
                    if (loads) mbar_arrive_expect_tx(&sh.full[st], (uint32_t)(g1 - c0) * 16);
                    else mbar_arrive(&sh.full[st]);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {
            atomicOr(P.err, ERR_TIMEOUT_EMPTY);
            sh.dead = 1;
        }
    } else {  // ---- the teams
        const int team = tid / TEAM, t = tid % TEAM;
        int turn = 0;  // counts the team's rows that are not ignored
        for (long long n = team; n < count; n += TEAMS) {
            const int st = (int)(n % stages);
            // A wait that runs out is noted, and the warp goes to the team's next barrier, after
            // which the whole team leaves.
            StageWait<RingShared<TEAMS>> wait{sh, st};
            StageInputs in;
            if (!take_row(wait, n, stages, in)) {
                if (t % 32 == 0) atomicOr(P.err, ERR_TIMEOUT_FULL);
                *(volatile int *)&sh.dead = 1;
                team_any<TEAM>(team, true);
                break;
            }
            const StageRow &at_stage = sh.row[st];
            const PolicyRow q = in.q;
            const float ref = in.ref, z_t = in.z_t;
            const long long row = in.row;
            char *out = P.dlogits + row * P.ld_d_bytes;
            const char *z = P.in.logits + row * P.in.ld_bytes;
            if (q.target < 0) {
                __syncwarp();
                if (t % 32 == 0) mbar_arrive(&sh.empty[st]);
                if (rank == 0 && t == 0) ignore_row(P, row);
                zero_row<DT>(out, P.in.vocab, rank * TEAM + t, cs * TEAM);
                if (team_any<TEAM>(team, *(volatile int *)&sh.dead != 0)) break;
                continue;
            }
            const Row<DT> r(z, P.in.vocab);
            int c0, g1;
            run_of(r, c0, g1);
            const int G = g1 - c0;
            const uint4 *stage = (const uint4 *)(ring + (size_t)st * stage_bytes);
            const int at = rank != 0 ? -1 : t == 0 && r.has_front() ? 0 : t == 1 && r.has_back() ? r.end() : -1;
            const uint4 edge = at >= 0 ? at_stage.edge[t] : Row<DT>::none();  // (t is 0 or 1)
            auto best = Elem<DT>::raise(Elem<DT>::lowest(), edge);
#pragma unroll 4
            for (int g = t; g < G; g += TEAM) best = Elem<DT>::raise(best, stage[g]);
            const Shift hw = shift_of<DT, ENT>(lanes_max(Elem<DT>::largest(best), 32), k);
            Sums<DT, ENT> sums = hw.ok ? stage_sums<DT, ENT, true, TEAM>(stage, t, G, hw)
                                            : stage_sums_slow<DT, ENT, TEAM>(stage, t, G, hw);
            if (at >= 0) {
                if (hw.ok) sums.template add<true>(edge, hw);
                else sums.template add<false>(edge, hw);
            }
            const Part mine = sums.part(hw, 32);
            const int b = turn & 1;
            if (t % 32 < cs)
                send_part(&sh.parts[team][b][rank * TEAM_WARPS + t / 32], &sh.joined[team][b], t % 32,
                          make_float4(mine.m, mine.s, mine.t, 0.f));
            if (t < 32) {
                if (t == 0) mbar_arrive_expect_tx(&sh.joined[team][b], cs * TEAM_WARPS * 16);
                if (__all_sync(ALL_LANES, mbar_wait(&sh.joined[team][b], turn >> 1 & 1))) {
                    const Part all = join_parts<ENT>(sh.parts[team][b], cs * TEAM_WARPS, k);
                    Terms terms{};
                    const Coef c = finish_row<ENT>(P, row, q, ref, all, z_t, rank == 0 && t == 0, terms);
                    if (t == 0) {
                        sh.coef[team][b] = c;
                        sh.sums[team].add(terms);
                    }
                } else {  // (the parts are not all there)
                    if (t == 0) atomicOr(P.err, ERR_TIMEOUT_ACC);
                    *(volatile int *)&sh.dead = 1;
                }
            }
            ++turn;
            if (team_any<TEAM>(team, *(volatile int *)&sh.dead != 0)) break;
            const Coef c = sh.coef[team][b];
            const Shift h = shift_of<DT, ENT>(c.m, k, c.b);
            if (c.none) {
                zero_row<DT>(out, P.in.vocab, rank * TEAM + t, cs * TEAM);
            } else if (!h.ok || (((uintptr_t)out ^ (uintptr_t)z) & 15) != 0) {
                grad_row_apart<DT, ENT>(z, out, P.in.vocab, q.target, z_t, c, k, rank * TEAM + t, cs * TEAM);
            } else {
                const Coef d = shifted(c, h);
                uint4 *o = (uint4 *)(out - r.phase * sizeof(typename Row<DT>::bits)) + c0;
#pragma unroll 4
                for (int g = t; g < G; g += TEAM) o[g] = grad_group<DT, ENT, true>(stage[g], d, h);
                if (at >= 0)
                    Row<DT>::store_edge(out, r.first(at), r.n, grad_group<DT, ENT, true>(at_stage.edge[t], d, h));
                // the thread that wrote the target's group adds its g
                const int tg = (q.target + r.phase) / Elem<DT>::N;
                if (tg == at || (tg >= c0 && tg < g1 && (tg - c0) % TEAM == t))
                    ((typename Row<DT>::bits *)out)[q.target] = Elem<DT>::round(grad_target<ENT>(z_t, c, k));
            }
            __syncwarp();
            if (t % 32 == 0) mbar_arrive(&sh.empty[st]);
        }
    }
    __syncthreads();
    const bool dead = sh.dead != 0;
    if (dead && tid == 0)  // copies in flight land before the CTA leaves
        for (int i = 0; i < stages; ++i) {
            StageWait<RingShared<TEAMS>> wait{sh, i, 100000000ull};
            drain_stage(wait, stages);
        }
    // no CTA leaves while others may still write into its shared memory
    cluster_sync();
    if (dead && tid == 0) {  // (parts that were sent here and that no wait has seen: far less than 1 ms)
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {}
    }
    if (rank != 0) return;
    TermSums sums = sh.sums[0];
    for (int i = 1; i < TEAMS; ++i) sums.add(sh.sums[i]);
    leave_sums(P, sums, (int)first, (int)step);
}

// ------------------------------------------------------------ gradient

struct GradParams {
    LogitsIn in;
    long long rows;
    const float2 *ms;       // (m, s) of each row
    const float *entropy;   // with gh
    const float *g, *gh;    // gradients of logp and H (gh may be null), gs apart
    int gs;
    float scale;            // the call's scale / tau
    char *out;
    long long ld_out_bytes;
};

// The gradient from saved statistics: one read of the logits, one write, no reduction
// and no barrier.  T threads of a block of THREADS to a row: all of them, or fewer where
// rows are short.  Rows are taken from the last: the statistics' launch has left the last
// of the logits in the L2 cache (126 MB at most).
// 12000 x 128000 bf16 (5.2 GB, 30% of the rows zeros) takes 770 us, 6.8 TB/s; 6000 x 32000
// with an entropy's gradient (730 MB) 110 us, 6.6 TB/s.
template <int DT, bool ENT, int T>
__global__ void __launch_bounds__(THREADS) grad_kernel(const __grid_constant__ GradParams P) {
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % T;
    // from the last row: what the statistics have read last is still in the L2 cache
    for (long long row = P.rows - 1 - ((long long)blockIdx.x * (THREADS / T) + threadIdx.x / T); row >= 0;
         row -= (long long)gridDim.x * (THREADS / T)) {
        const long long tgt = target_of(P.in, row);
        const float2 ms = P.ms[row];
        const Coef c = coef_of<ENT>(ms.x, ms.y, ENT ? P.entropy[row] : 0.f, P.g[row * P.gs] * P.scale,
                                    ENT ? P.gh[row * P.gs] * P.scale : 0.f);
        char *out = P.out + row * P.ld_out_bytes;
        if (tgt < 0 || tgt >= P.in.vocab || c.none)
            zero_row<DT>(out, P.in.vocab, t, T);
        else {
            const char *z = P.in.logits + row * P.in.ld_bytes;
            grad_row<DT, ENT>(z, out, P.in.vocab, (int)tgt, logit_at<DT>(z, tgt), c, P.in.k, t, T);
        }
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

struct PolicyRows {
    LogitsIn in;
    long long rows;
    const float *weight, *advantage, *old_logp;
    const int32_t *off;
    int seqs, seq_mean;
    PolicyRow *meta;
    int *order;  // may be null
    unsigned *done;
    int *err;
};

// A row of the policy loss from the caller's arrays (weight 1 where none is given).
__device__ __forceinline__ PolicyRow policy_row(const PolicyRows &P, long long row, int &bad) {
    const long long t = target_of(P.in, row);
    bad |= t >= P.in.vocab;
    const int seq = P.off ? sequence_of(P.off, P.seqs + 1, row) : 0;
    const float w = P.weight ? P.weight[row] : 1.f;
    PolicyRow q{-1, 0.f, 0.f, 0.f};
    if (t >= 0 && t < P.in.vocab && w != 0.f && seq >= 0 && (!P.off || seq < P.seqs))
        q = PolicyRow{(int)t, w, P.advantage[P.off ? seq : row], P.old_logp[row]};
    return q;
}

constexpr int SMALL_CLUSTER = 8, ROWS_THREADS = 512;

// The whole policy loss of few short rows in one cluster: every CTA counts the
// rows for itself (where the weight is one over their number), its groups of lanes
// take the rows in turn, and the terms are added up across the cluster.  One
// launch in place of three, each of which would take longer to start than to run:
// a call on 100 x 1000 fp32 takes 35 us in three launches, 30 in this form.
// Up to SMALL_ROUNDS rows to a group: at 2000 x 18 the GPU needs 22 us either way; with
// 16 rounds 6000 x 18 takes 45 us here and 22 in three launches.  The preference loss takes
// the same bound.  Its calls are bound by the host there, where one launch is the shorter
// (500 x 1000 fp32: 31 us a call, 41 in three launches; 2000 x 200: 32 and 41), though the
// GPU alone would need less in three (35 us against 28 for both, as a captured graph
// sees it); with 16 rounds 1500 x 1000 takes 69 us a call in place of 40.
constexpr int SMALL_ROUNDS = 4;
template <int DT, bool ENT, int L>
__global__ void __launch_bounds__(ROWS_THREADS) policy_small_kernel(const __grid_constant__ RowParams P,
                                                                    const __grid_constant__ PolicyRows R, float *stats) {
    __shared__ int part[32];
    cluster_arrive();
    pdl_wait();
    pdl_trigger();
    int n = 0, bad = 0;
    for (long long row = threadIdx.x; row < R.rows; row += ROWS_THREADS) {
        const long long t = target_of(R.in, row);
        bad |= t >= R.in.vocab;
        n += t >= 0 && t < R.in.vocab && (!R.off || (row >= R.off[0] && row < R.off[R.seqs]));
    }
    n = block_sum(n, part);
    bad = __syncthreads_or(bad);
    const float w = 1.f / (float)n;
    TermSums sums{};
    constexpr int PER = ROWS_THREADS / L;
    for (long long first = (long long)blockIdx.x * PER + threadIdx.x / 32 * (32 / L); first < R.rows;
         first += (long long)gridDim.x * PER) {
        const long long row = first + threadIdx.x % 32 / L;
        PolicyRow q{-1, 0.f, 0.f, 0.f};
        int unused = 0;
        if (row < R.rows) q = policy_row(R, row, unused);
        if (!R.weight) q.weight = w;
        const Terms o = lane_row<DT, ENT, L>(P, row, row < R.rows, q);
        if (threadIdx.x % L == 0) sums.add(o);
    }
    __shared__ TermSums all[SMALL_CLUSTER];
    sums.add_block();
    cluster_wait();
    if (threadIdx.x == 0) {
        *peer(&all[blockIdx.x], 0) = sums;
        if (blockIdx.x == 0) *R.err = bad ? ERR_TARGET : 0;
    }
    cluster_sync();
    if (blockIdx.x != 0 || threadIdx.x != 0) return;
    for (int c = 1; c < (int)gridDim.x; ++c) sums.add(all[c]);
    sums.write(stats, R.err, 0);
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
    float scale;         // the call's scale / tau (0 for a call without gradient)
    const float *logp;   // of every row (0 where ignored)
    const float2 *ms;
    float *row_g;        // gradient of every row's logp
    float *terms;        // [pairs] weighted f
    int *bad;            // [pairs] error bits
    float *pair_loss, *seq_logp;
};

// ln(1 + e^-x) = -ln sigma(x) without overflow.
__device__ __forceinline__ float softplus_neg(float x) { return fmaxf(-x, 0.f) + log1pf(expf(-fabsf(x))); }

// The sums of a pair's two sequences, f and its derivative, by a team of T
// threads (a warp or a block).  h is formed in more than fp32 (two sums that nearly
// cancel), f from it in fp32.  (What other CTAs have written is read past L1.)
constexpr int PAIR_THREADS = 256;
template <int T>
__device__ __forceinline__ void pref_pair(const PrefPairs &P, int b) {
    __shared__ Wide part[32];
    __shared__ int ipart[32], ibad[16];
    __shared__ float shared_slope[2];
    const int t = threadIdx.x % T;
    long long r0[2], r1[2];
    double l[2] = {0., 0.};
    Wide sum[2] = {};
    int n[2] = {0, 0}, bad = 0;
    const long long cut = clamp_row(P.off[2 * b + 1], P.rows);
    r0[0] = clamp_row(P.off[2 * b], P.rows);
    r1[0] = r0[1] = cut;
    r1[1] = clamp_row(P.off[2 * b + 2], P.rows);
    for (int q = 0; q < 2; ++q) {
        for (long long row = r0[q] + t; row < r1[q]; row += T) {
            const long long tg = P.target_i32 ? (long long)((const int32_t *)P.target)[row]
                                              : (long long)((const int64_t *)P.target)[row];
            if (tg >= P.vocab) bad |= ERR_TARGET;
            if (tg < 0 || tg >= P.vocab) continue;
            ++n[q];
            if (__ldcg(&P.ms[row].y) == 0.f) {  // every logit -inf: left out
                bad |= ERR_NONFINITE;
                continue;
            }
            const float v = __ldcg(&P.logp[row]);
            if (!finite(v)) bad |= ERR_NONFINITE;
            sum[q].add(v);
        }
    }
    for (int q = 0; q < 2; ++q) {
        sum[q].add_lanes();
        n[q] = __reduce_add_sync(0xffffffffu, n[q]);
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if constexpr (T > 32) {
        constexpr int W = T / 32;
        if (threadIdx.x % 32 == 0) {
            const int w = threadIdx.x / 32;
            part[w] = sum[0];
            part[W + w] = sum[1];
            ipart[w] = n[0];
            ipart[W + w] = n[1];
            ibad[w] = bad;
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            for (int q = 0; q < 2; ++q) {
                sum[q] = threadIdx.x < W ? part[q * W + threadIdx.x] : Wide{};
                sum[q].add_lanes();
                n[q] = __reduce_add_sync(0xffffffffu, threadIdx.x < W ? ipart[q * W + threadIdx.x] : 0);
            }
            bad = __reduce_or_sync(0xffffffffu, threadIdx.x < W ? ibad[threadIdx.x] : 0);
        }
    }
    if (t == 0)
        for (int q = 0; q < 2; ++q) {
            const Wide s = sum[q];
            l[q] = P.average && n[q] > 0 ? s.value() / n[q] : s.value();
            if (!finite((float)l[q])) bad |= ERR_NONFINITE;
            if (P.seq_logp) P.seq_logp[2 * b + q] = (float)l[q];
        }
    float slope[2] = {0.f, 0.f};
    if (t == 0) {
        double h = l[0] - l[1];
        if (P.ref) h -= (double)P.ref[2 * b] - (double)P.ref[2 * b + 1];
        const float beta = P.beta, e = P.smooth, x = (float)(beta * h);
        float f, d;
        if (P.kind == KFAC_PREF_SIGMOID) {
            f = (1.f - e) * softplus_neg(x) + (e > 0.f ? e * softplus_neg(-x) : 0.f);
            d = beta * ((e > 0.f ? e / (1.f + expf(-x)) : 0.f) - (1.f - e) / (1.f + expf(x)));
        } else if (P.kind == KFAC_PREF_HINGE) {
            f = x < 1.f ? (float)(1. - beta * h) : x >= 1.f ? 0.f : x;  // (NaN stays)
            d = x < 1.f ? -beta : x >= 1.f ? 0.f : x;
        } else {
            const float o = (float)(h - 0.5 / beta);
            f = o * o;
            d = 2.f * o;
        }
        const float v = P.pair_weight ? P.pair_weight[b] : 1.f / (float)P.pairs;
        if (!finite(f)) bad |= ERR_NONFINITE;
        P.terms[b] = v == 0.f ? 0.f : v * f;
        if (P.pair_loss) P.pair_loss[b] = f;
        for (int q = 0; q < 2; ++q) {
            slope[q] = v == 0.f ? 0.f : v * d * (q ? -1.f : 1.f) / (P.average && n[q] > 0 ? (float)n[q] : 1.f);
            if (P.scale != 0.f && n[q] > 0 && !finite(slope[q] * P.scale)) bad |= ERR_NONFINITE;
            if (T > 32) shared_slope[q] = slope[q];
        }
    }
    if constexpr (T > 32) {
        __syncthreads();
        slope[0] = shared_slope[0];
        slope[1] = shared_slope[1];
    } else {
        slope[0] = __shfl_sync(0xffffffffu, slope[0], 0);
        slope[1] = __shfl_sync(0xffffffffu, slope[1], 0);
    }
    if (t == 0) P.bad[b] = bad;
    for (int q = 0; q < 2; ++q)
        for (long long row = r0[q] + t; row < r1[q]; row += T) P.row_g[row] = slope[q];
}

struct PrefSum {
    const float *terms;
    const int *bad;
    int pairs;
    float *loss;
    int *err;
    unsigned *done;  // CTAs that have finished their pair
};
// The loss over all pairs, by one block, in a fixed order.
__device__ __forceinline__ void pref_sum(const PrefSum &P) {
    __shared__ Wide part[32];
    __shared__ int ipart[32];
    Wide s{};
    int bad = 0;
    for (int b = threadIdx.x; b < P.pairs; b += blockDim.x) {
        s.add(__ldcg(&P.terms[b]));
        bad |= __ldcg(&P.bad[b]);
    }
    s = block_sum(s, part);
    const int nf = block_sum(bad & ERR_NONFINITE ? 1 : 0, ipart), tg = block_sum(bad & ERR_TARGET ? 1 : 0, ipart);
    if (threadIdx.x == 0) {
        const float loss = (float)s.value();
        *P.loss = loss;
        *P.err = (nf || !finite(loss) ? ERR_NONFINITE : 0) | (tg ? ERR_TARGET : 0);
    }
}

// The whole preference loss of few short rows in one cluster: rows, then pairs,
// then the rows' gradients, with a cluster barrier after each (a call on
// two pairs of 97 rows x 1000 fp32 takes 41 us in four launches, 33 in this form).
template <int DT, int L>
__global__ void __launch_bounds__(ROWS_THREADS) pref_small_kernel(const __grid_constant__ RowParams P,
                                                                  const __grid_constant__ PrefPairs Q,
                                                                  const __grid_constant__ PrefSum U, char *dlogits) {
    pdl_wait();
    pdl_trigger();
    constexpr int PER = ROWS_THREADS / L;
    const long long start = (long long)blockIdx.x * PER + threadIdx.x / 32 * (32 / L), step = (long long)gridDim.x * PER;
    for (long long first = start; first < P.rows; first += step) {
        const long long row = first + threadIdx.x % 32 / L;
        PolicyRow q{-1, 0.f, 0.f, 0.f};
        if (row < P.rows) q = row_meta(P, row);
        lane_row<DT, false, L>(P, row, row < P.rows, q);
    }
    cluster_sync();
    for (int b = blockIdx.x * (ROWS_THREADS / 32) + threadIdx.x / 32; b < Q.pairs; b += gridDim.x * (ROWS_THREADS / 32))
        pref_pair<32>(Q, b);
    cluster_sync();
    if (blockIdx.x == 0) pref_sum(U);
    if (!dlogits) return;
    const int lane = threadIdx.x % L;
    for (long long first = start; first < P.rows; first += step) {
        const long long row = first + threadIdx.x % 32 / L;
        if (row >= P.rows) continue;
        const PolicyRow q = row_meta(P, row);
        const char *z = P.in.logits + row * P.in.ld_bytes;
        char *out = dlogits + row * P.ld_d_bytes;
        const float2 ms = __ldcg(&P.ms[row]);
        const Coef c = coef_of<false>(ms.x, ms.y, 0.f, __ldcg(&Q.row_g[row]) * P.scale, 0.f);
        if (q.target < 0 || c.none) zero_row<DT>(out, P.in.vocab, lane, L);
        else grad_row<DT, false>(z, out, P.in.vocab, q.target, logit_at<DT>(z, q.target), c, P.in.k, lane, L);
    }
}

// ------------------------------------------------------------ launches

// How rows are kept in shared memory: by how many CTAs, in how many stages.
struct Ring {
    int cs, stages, bytes, teams;  // cs = 0: they do not fit
};
inline Ring ring_of(int dtype, int vocab, long long rows) {
    const long long whole = vocab / (dtype == KFAC_F32 ? 4 : 8);  // whole groups of a row, at most
    Ring g{1, 0, 0, 2};
    auto bytes = [&](int cs) { return ceil_div(whole, cs) * 16; };
    // Three stages at least, for which a row goes to up to four CTAs: 2000 x 50001 takes
    // 94 us in two stages of one CTA, 89 in four stages of two.  Eight CTAs only where two
    // stages would not fit otherwise: 1500 x 200000 takes 274 us by eight, 235 by four in
    // two stages.
    while (g.cs < MAX_CLUSTER / 2 && bytes(g.cs) > RING_BYTES / 3) g.cs *= 2;
    while (g.cs < MAX_CLUSTER && bytes(g.cs) > RING_BYTES / 2) g.cs *= 2;
    // few rows: more CTAs to each, while a thread has two groups
    while (g.cs < MAX_CLUSTER && rows * g.cs * 2 <= device_sm_count() && whole >= (long long)g.cs * 1024) g.cs *= 2;
    if (bytes(g.cs) > RING_BYTES / 2) return Ring{0, 0, 0, 0};
    g.bytes = (int)align_up((size_t)bytes(g.cs), 128);
    // Shorter runs, more and smaller teams (the fixed work of a row is then shared out):
    // 8000 x 8200 takes 107 us by two teams, 75 by four, 61 by eight; 6000 x 20000 takes
    // 92 by four and 100 by eight, 4000 x 16001 in fp32 95 by two and 107 by four.
    g.teams = bytes(g.cs) > 3500 * 16 ? 2 : bytes(g.cs) > 1536 * 16 ? 4 : 8;
    g.stages = (int)std::min<long long>(MAX_STAGES, RING_BYTES / std::max(g.bytes, 128));
    return g;
}

// CTAs (clusters) of a launch over rows, at most: each leaves its sums.
constexpr int MAX_CTAS = 1 << 14;

// Whether rows go to warps: a CTA's barriers cost more than a second pass over short
// rows.  Statistics of 8000 x 6000 bf16 (750 groups) take 24 us by warps and 35 by CTAs, of
// 8000 x 8192 28 and 36.  With the gradient 16000 x 2100 takes 60 us by warps and 86 in the
// ring, 8000 x 4096 47 and 46, 8000 x 6000 70 and 52.  Fewer rows than SMs leave warps idle
// unless they are very short.
inline bool by_warps(long long whole, long long rows, bool gradient) {
    return whole <= WARP_SHORT ||
           (whole <= (gradient ? WARP_GRAD_GROUPS : WARP_GROUPS) && rows >= device_sm_count());
}

struct RunRows {
    const RowParams &P;
    cudaStream_t st;
    template <int DT, bool ENT, int TEAMS>
    kfac_status ring(const Ring &g) {
        auto kernel = ring_rows_kernel<DT, ENT, TEAMS>;
        static std::atomic<int> ready[64][4];  // by device and cluster size: clusters that run at once
        int dev = 0, lg = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KFAC_ERR_CUDA;
        while ((1 << lg) < g.cs) ++lg;
        int most = ready[dev][lg].load(std::memory_order_relaxed);
        if (most == 0) {
            KFAC_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES));
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(device_sm_count() / g.cs * g.cs);
            cfg.blockDim = dim3(RING_THREADS);
            cfg.dynamicSmemBytes = RING_BYTES;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = g.cs;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            KFAC_CUDA_TRY(cudaOccupancyMaxActiveClusters(&most, kernel, &cfg));
            if (most < 1) return KFAC_ERR_CUDA;
            ready[dev][lg].store(most, std::memory_order_relaxed);
        }
        const unsigned grid = (unsigned)std::min<long long>(P.rows, most) * g.cs;
        KFAC_LAUNCH_CLUSTERS(KK_LOSS_ROWS, st, kernel, g.cs, grid, RING_THREADS, (size_t)g.stages * g.bytes, P, g.cs,
                             g.stages, g.bytes);
        return KFAC_OK;
    }
    template <int DT, bool ENT>
    kfac_status run() {
        const long long whole = P.in.vocab / Elem<DT>::N;
        if (by_warps(whole, P.rows, P.dlogits)) {
            const int L = lanes_of(whole, P.rows);
            const unsigned grid = (unsigned)std::min<long long>(ceil_div(P.rows, WARP_THREADS / L),
                                                                device_sm_count() * WARP_PER_SM);
            if (L == 8) KFAC_LAUNCH(KK_LOSS_ROWS, st, (warp_rows_kernel<DT, ENT, 8>), grid, WARP_THREADS, 0, P);
            else if (L == 16) KFAC_LAUNCH(KK_LOSS_ROWS, st, (warp_rows_kernel<DT, ENT, 16>), grid, WARP_THREADS, 0, P);
            else KFAC_LAUNCH(KK_LOSS_ROWS, st, (warp_rows_kernel<DT, ENT, 32>), grid, WARP_THREADS, 0, P);
            return KFAC_OK;
        }
        const Ring g = P.dlogits ? ring_of(DT, P.in.vocab, P.rows) : Ring{0, 0, 0, 0};
        if (g.cs) return g.teams == 2 ? ring<DT, ENT, 2>(g) : g.teams == 4 ? ring<DT, ENT, 4>(g) : ring<DT, ENT, 8>(g);
        // few rows: more CTAs to each, while there is room and a thread has two groups
        int cs = 1;
        while (cs < MAX_CLUSTER && P.rows * cs < device_sm_count() * STREAM_PER_SM &&
               whole >= (long long)cs * STREAM_THREADS * 4)
            cs *= 2;
        const unsigned grid = (unsigned)std::min<long long>(P.rows, MAX_CTAS) * cs;
        KFAC_LAUNCH_CLUSTERS(KK_LOSS_ROWS, st, (stream_rows_kernel<DT, ENT>), cs, grid, STREAM_THREADS, 0, P, cs);
        return KFAC_OK;
    }
};
// Lanes to a row of the small kernels (0: the call is not one of few short rows).
inline int small_lanes(int dtype, int vocab, long long rows) {
    const long long whole = vocab / (dtype == KFAC_F32 ? 4 : 8);
    const int L = whole <= 8 * NV ? 8 : whole <= 32 * NV ? 32 : 0;
    return L && rows * L <= SMALL_ROUNDS * SMALL_CLUSTER * ROWS_THREADS ? L : 0;
}
inline unsigned small_ctas(int L, long long rows) {
    unsigned n = 1;
    while (n < SMALL_CLUSTER && (long long)n * (ROWS_THREADS / L) < rows) n *= 2;
    return n;
}
struct RunPolicySmall {
    const RowParams &P;
    const PolicyRows &R;
    float *stats;
    int L;
    cudaStream_t st;
    template <int DT, bool ENT>
    kfac_status run() {
        const unsigned n = small_ctas(L, R.rows);
        if (L == 8)
            KFAC_LAUNCH_CLUSTERS(KK_LOSS_ROWS, st, (policy_small_kernel<DT, ENT, 8>), n, n, ROWS_THREADS, 0, P, R, stats);
        else
            KFAC_LAUNCH_CLUSTERS(KK_LOSS_ROWS, st, (policy_small_kernel<DT, ENT, 32>), n, n, ROWS_THREADS, 0, P, R, stats);
        return KFAC_OK;
    }
};
struct RunPrefSmall {
    const RowParams &P;
    const PrefPairs &Q;
    const PrefSum &U;
    char *dlogits;
    int L;
    cudaStream_t st;
    template <int DT, bool>
    kfac_status run() {
        const unsigned n = small_ctas(L, P.rows);
        if (L == 8)
            KFAC_LAUNCH_CLUSTERS(KK_LOSS_ROWS, st, (pref_small_kernel<DT, 8>), n, n, ROWS_THREADS, 0, P, Q, U, dlogits);
        else
            KFAC_LAUNCH_CLUSTERS(KK_LOSS_ROWS, st, (pref_small_kernel<DT, 32>), n, n, ROWS_THREADS, 0, P, Q, U, dlogits);
        return KFAC_OK;
    }
};
struct RunGrad {
    const GradParams &P;
    cudaStream_t st;
    template <int DT, bool ENT>
    kfac_status run() {
        const long long whole = P.in.vocab / Elem<DT>::N;
        const int L = lanes_of(whole, P.rows);
        const unsigned grid = (unsigned)std::min<long long>(ceil_div(P.rows, THREADS / L), 1 << 20);
        if (whole <= WARP_GROUPS && L < 32)
            KFAC_LAUNCH(KK_LOSS_GRAD, st, (grad_kernel<DT, ENT, 8>), (unsigned)std::min<long long>(ceil_div(P.rows, THREADS / 8), 1 << 20), THREADS, 0, P);
        else if (whole <= WARP_GROUPS)
            KFAC_LAUNCH(KK_LOSS_GRAD, st, (grad_kernel<DT, ENT, 32>), grid, THREADS, 0, P);
        else
            KFAC_LAUNCH(KK_LOSS_GRAD, st, (grad_kernel<DT, ENT, THREADS>),
                        (unsigned)std::min<long long>(P.rows, 1 << 20), THREADS, 0, P);
        return KFAC_OK;
    }
};

// One call's launches for logits of type DT, each type's in a source file of its own.
template <int DT>
kfac_status launch_rows(const RowParams &P, bool ent, cudaStream_t st) {
    RunRows r{P, st};
    return ent ? r.run<DT, true>() : r.run<DT, false>();
}
template <int DT>
kfac_status launch_grad(const GradParams &P, bool ent, cudaStream_t st) {
    RunGrad r{P, st};
    return ent ? r.run<DT, true>() : r.run<DT, false>();
}
template <int DT>
kfac_status launch_policy_small(const RowParams &P, const PolicyRows &R, float *stats, int L, bool ent, cudaStream_t st) {
    RunPolicySmall r{P, R, stats, L, st};
    return ent ? r.run<DT, true>() : r.run<DT, false>();
}
template <int DT>
kfac_status launch_pref_small(const RowParams &P, const PrefPairs &Q, const PrefSum &U, char *dlogits, int L,
                              cudaStream_t st) {
    RunPrefSmall r{P, Q, U, dlogits, L, st};
    return r.run<DT, false>();
}
#define KFAC_LOSS_LAUNCHES(PREFIX, DT)                                                                              \
    PREFIX template kfac_status launch_rows<DT>(const RowParams &, bool, cudaStream_t);                             \
    PREFIX template kfac_status launch_grad<DT>(const GradParams &, bool, cudaStream_t);                            \
    PREFIX template kfac_status launch_policy_small<DT>(const RowParams &, const PolicyRows &, float *, int, bool,  \
                                                        cudaStream_t);                                              \
    PREFIX template kfac_status launch_pref_small<DT>(const RowParams &, const PrefPairs &, const PrefSum &, char *, \
                                                      int, cudaStream_t);

}  // namespace loss
}  // namespace kfac
