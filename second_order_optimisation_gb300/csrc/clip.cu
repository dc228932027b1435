// clip.cu -- kfac_clip_norm: the norm over many tensors, clipping, and the
// step on the weights.
//
//   norm = sqrt(sum x y)  (y = x: the Euclidean norm),  scale = min(1, max_norm / norm),
//   out = scale x,  w <- w - eta scale x.
//
// Bound by memory: x (and y) are read for the norm, x (and w) again for the
// step.  The tensors are cut into octets of eight elements, numbered through all
// tensors, and every CTA takes an equal run of them in both passes; the second
// pass walks its run from the end, so that what the first has read last is still
// in the L2 cache.  A thread adds up to 64 products in fp32 (16-bit x without y; 32
// otherwise) and those sums in two fp32 words; the CTAs' sums are added in fp64 in a
// fixed order.  A run whose sum overflows or vanishes in fp32 is summed again from values
// scaled by a power of two, so that any finite input gives its norm.  (So is a run of
// zeros: eight 4096 x 4096 fp32 tensors of zeros take 540 us for the norm, 97 otherwise.)
//
// Measured: 48 tensors of 1.0e9 bf16 values, out on other 16-byte offsets than x: 312 us
// for the norm (2.0 GB, 6.5 TB/s), 651 for the scaling (4.0 GB, 6.2 TB/s); ResNet-50's 161
// fp32 tensors with metric and weight step: 45 us (204 MB, 4.5 TB/s) and 49 us (307 MB,
// 6.2 TB/s), the norm bound by the latency of the many runs that its first tiles hold.
// 256 threads, three CTAs to an SM: the scaling took 663 us so, 700 by 512 x 2, 771 by
// 256 x 4, 924 by 1024 x 2 (fewer streams open at once suit the memory better).
// Tensors with gaps between their rows go octet by octet through a division, and element
// by element where a pitch of any of their operands is not a multiple of eight elements:
// ResNet-50's layers as KfacStep keeps them (fp32 steps and bf16 gradients on pitches of 64
// elements, dense weights) take 59 and 124 us, 357 MB with a floor of 53; four layers of
// 4096 x 4097 159 and 403 us, floor 139.
#include <algorithm>
#include <cmath>
#include <memory>

#include "logits.cuh"

namespace kfac {
namespace {

constexpr int CLIP_FEW = 16, CLIP_MANY = 216;  // tensors of one launch (kernel parameters)
constexpr int CLIP_THREADS = 256, CLIP_PER_SM = 3, OCTET = 8, SHORT_RUN = 192, TILE = 4096, SMALL_OCTETS = 16384;
constexpr int CTA_OCTETS = 64;  // a CTA's least share
constexpr int LINE = 8;         // octets of 16-bit values in 128 bytes

struct ClipJob {
    const char *x, *y;
    char *out;
    float *w;
    long long ld, ld_y, ld_out, ld_w;
    long long rows, cols;  // a tensor without gaps is one row
    long long first;       // its first octet of the launch
    long long per_row;     // octets of a row
    uint8_t dtype, y_dtype, out_dtype;
    uint8_t shift;         // octet 0 starts this many elements before the row
    uint8_t vec;           // octets are taken 16 bytes at a time
    uint8_t out_vec;       // ... and stored so
};
template <int MAX>
struct ClipParams {
    ClipJob job[MAX];
    int n;
    long long octets, tile;
    double *part;        // one for each CTA of each launch
    int part0, parts;    // this launch's first, and all launches'
    float max_norm, eta;
    float *norm, *scale;
    int *err;            // set by the first launch of the second pass
};

template <int DT>
__device__ __forceinline__ float elem(const char *p, long long i) {
    return Elem<DT>::value(((const typename Elem<DT>::bits *)p)[i]);
}

// Eight elements from any element boundary.
template <int DT, bool ANY>
struct Raw : Pieces<Elem<DT>::N == 4 ? 2 : 1, ANY> {
    static constexpr int Q = Elem<DT>::N == 4 ? 2 : 1;
    __device__ __forceinline__ void values(int off, float *v) const {
        uint4 w[Q];
        this->take(off, w);
#pragma unroll
        for (int q = 0; q < Q; ++q) Elem<DT>::unpack(w[q], v + 4 * q);
    }
};
template <int DT>
__device__ __forceinline__ void load8(const char *p, int off, float *v) {
    if (off == 0) {
        Raw<DT, false> r;
        r.load(p, off);
        r.values(off, v);
    } else {
        Raw<DT, true> r;
        r.load(p, off);
        r.values(off, v);
    }
}
template <int DT>
__device__ __forceinline__ void store8(char *p, const float *v) {
    constexpr int Q = Elem<DT>::N == 4 ? 2 : 1;
#pragma unroll
    for (int q = 0; q < Q; ++q) *reinterpret_cast<uint4 *>(p + 16 * q) = Elem<DT>::pack(v + 4 * q);
}

// Where octet i of a tensor lies: row, first column (may be negative), and
// whether all its elements, and eight on both sides, exist.
struct Place {
    long long row, col;
    bool whole, inner;
};
__device__ __forceinline__ Place place_of(const ClipJob &j, long long i) {
    Place p;
    p.row = 0;
    if (j.rows > 1) {
        p.row = j.rows * j.per_row <= 0xffffffffLL ? (long long)((uint32_t)i / (uint32_t)j.per_row) : i / j.per_row;
        i -= p.row * j.per_row;
    }
    p.col = i * OCTET - j.shift;
    p.whole = p.col >= 0 && p.col + OCTET <= j.cols;
    p.inner = p.col >= OCTET && p.col + 2 * OCTET <= j.cols;
    return p;
}
template <int DT>
__device__ __forceinline__ void octet(const char *base, long long ld, const Place &p, long long cols, bool vec, float *v) {
    constexpr int ES = Elem<DT>::N == 4 ? 4 : 2;
    const char *row = base + p.row * ld * ES, *at = row + p.col * ES;
    const int off = (int)((uintptr_t)at & 15);
    if (vec && (p.inner || (p.whole && off == 0))) {
        load8<DT>(at, off, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < OCTET; ++e) v[e] = p.col + e >= 0 && p.col + e < cols ? elem<DT>(row, p.col + e) : 0.f;
}

template <class P>
__device__ __forceinline__ int job_of(const P &p, long long i) {
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.job[mid].first <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ Wide block_wide(Wide v) {
    __shared__ Wide part[CLIP_THREADS / 32];
    v.add_lanes();
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = threadIdx.x % 32 < CLIP_THREADS / 32 ? part[threadIdx.x % 32] : Wide{};
    v.add_lanes();
    return v;
}
__device__ __forceinline__ unsigned block_max(unsigned v) {
    __shared__ unsigned part[CLIP_THREADS / 32];
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = threadIdx.x % 32 < CLIP_THREADS / 32 ? part[threadIdx.x % 32] : 0;
    return __reduce_max_sync(0xffffffffu, v);
}

// The types of a tensor's x and y (NO_Y: there is none), as template arguments.
constexpr int NO_Y = -1;
template <int DT_, int YT_>
struct Types {
    static constexpr int DT = DT_, YT = YT_;
};
template <class F>
__device__ __forceinline__ auto by_types(const ClipJob &j, F &&f) {
    if (j.dtype == KFAC_BF16) return j.y ? f(Types<KFAC_BF16, KFAC_BF16>{}) : f(Types<KFAC_BF16, NO_Y>{});
    if (j.dtype == KFAC_F16) return j.y ? f(Types<KFAC_F16, KFAC_F16>{}) : f(Types<KFAC_F16, NO_Y>{});
    if (!j.y) return f(Types<KFAC_F32, NO_Y>{});
    return j.y_dtype == KFAC_BF16 ? f(Types<KFAC_F32, KFAC_BF16>{})
           : j.y_dtype == KFAC_F16 ? f(Types<KFAC_F32, KFAC_F16>{}) : f(Types<KFAC_F32, KFAC_F32>{});
}

// 2^n as fp32, n in -126 .. 127.
__device__ __forceinline__ float pow2(int n) { return __int_as_float((n + 127) << 23); }
// A power of two (as its exponent) that brings the largest magnitude (its bits) near 1.
__device__ __forceinline__ int to_one(unsigned magnitude) {
    return max(-126, min(126, 127 - (int)(magnitude >> 23)));
}

// The octets of lo .. hi - 1 of a tensor without gaps that have eight elements on
// both sides: they are taken from moving pointers, with no test of each.
__device__ __forceinline__ void inner_run(const ClipJob &j, long long lo, long long hi, long long &a, long long &b) {
    a = b = lo;
    if (j.rows > 1 || !j.vec) return;
    a = max(lo, (long long)(2 * OCTET + j.shift - 1) / OCTET);
    b = max(a, min(hi, (j.cols + j.shift) / OCTET - 1));
    if (a >= hi) a = b = lo;
}
__device__ __forceinline__ float sum_of_products(const float *x, const float *y) {
    float q[OCTET];
#pragma unroll
    for (int e = 0; e < OCTET; ++e) q[e] = x[e] * y[e];
    return ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
}
template <int DT, int YT, bool ANY>
__device__ __noinline__ Wide inner_products(const ClipJob &j, long long a, long long b, Wide sum) {
    constexpr bool METRIC = YT != NO_Y;
    constexpr int ES = Elem<DT>::N == 4 ? 4 : 2, UNROLL = (METRIC ? 2 : 4) * (ES == 2 ? 2 : 1), STEP = CLIP_THREADS * OCTET * ES;
    constexpr int Y = METRIC ? YT : DT, ESY = Elem<Y>::N == 4 ? 4 : 2, STEPY = CLIP_THREADS * OCTET * ESY;
    const char *x = j.x + (a * OCTET - j.shift) * ES + threadIdx.x * (OCTET * ES);
    const char *y = METRIC ? j.y + (a * OCTET - j.shift) * ESY + threadIdx.x * (OCTET * ESY) : x;
    const int oy = (int)((uintptr_t)y & 15);  // (x is on its boundaries)
    long long left = b - a - threadIdx.x;  // octets from this thread's on
    for (; left > (UNROLL - 1) * CLIP_THREADS; left -= UNROLL * CLIP_THREADS) {
        Raw<DT, false> u[UNROLL];
        Raw<Y, ANY> v[METRIC ? UNROLL : 1];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            u[k].load(x + k * STEP, 0);
            if (METRIC) v[k].load(y + k * STEPY, oy);
        }
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            float f[OCTET], h[OCTET];
            u[k].values(0, f);
            if (METRIC) v[k].values(oy, h);
            t += sum_of_products(f, METRIC ? h : f);
        }
        sum.add(t);
        x += UNROLL * STEP;
        y += UNROLL * STEPY;
    }
    for (; left > 0; left -= CLIP_THREADS) {
        float f[OCTET], h[OCTET];
        load8<DT>(x, 0, f);
        if (METRIC) load8<Y>(y, oy, h);
        sum.add(sum_of_products(f, METRIC ? h : f));
        x += STEP;
        y += STEPY;
    }
    return sum;
}

template <int DT, int YT>
__device__ __noinline__ Wide outer_products(const ClipJob &j, long long lo, long long hi, int tid, int nt, Wide sum);
// This thread's sum of x y over octets lo .. hi - 1 of a tensor, added to `sum`.
// A short run, and a long one's ends, are one warp's, the n-th of them the
// n-th warp's, so that many small tensors go on side by side.  (100 tensors of 11 M
// fp16 values, with their metric, took 44 us; with SHORT_RUN = 48 47, with 1024 83.)
template <int DT, int YT>
__device__ __forceinline__ void products(const ClipJob &j, int n, long long lo, long long hi, Wide &sum) {
    const int lane = threadIdx.x % 32;
    const bool mine = (int)threadIdx.x / 32 == n % (CLIP_THREADS / 32);
    if (hi - lo < SHORT_RUN) {
        if (mine) sum = outer_products<DT, YT>(j, lo, hi, lane, 32, sum);
        return;
    }
    long long a, b;
    inner_run(j, lo, hi, a, b);
    if (b > a) {
        if (mine) sum = outer_products<DT, YT>(j, lo, a, lane, 32, sum);
        if (mine) sum = outer_products<DT, YT>(j, b, hi, lane, 32, sum);
        constexpr int ESY = YT == KFAC_F32 ? 4 : 2;
        if (YT != NO_Y && (((uintptr_t)j.y - (uintptr_t)j.shift * ESY) & 15))
            sum = inner_products<DT, YT, YT != NO_Y>(j, a, b, sum);
        else
            sum = inner_products<DT, YT, false>(j, a, b, sum);
    } else {
        sum = outer_products<DT, YT>(j, lo, hi, threadIdx.x, CLIP_THREADS, sum);
    }
}
template <int DT, int YT>
__device__ __noinline__ Wide outer_products(const ClipJob &j, long long lo, long long hi, int tid, int nt, Wide sum) {
    constexpr bool METRIC = YT != NO_Y;
    constexpr int Y = METRIC ? YT : DT, UNROLL = METRIC ? 2 : 4;  // octets in flight
    for (long long i = lo + tid; i < hi; i += UNROLL * nt) {
        float x[UNROLL][OCTET], y[UNROLL][OCTET];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const long long at = i + u * nt;
            if (at < hi) {
                const Place p = place_of(j, at);
                octet<DT>(j.x, j.ld, p, j.cols, j.vec, x[u]);
                if (METRIC) octet<Y>(j.y, j.ld_y, p, j.cols, j.vec, y[u]);
            } else {
#pragma unroll
                for (int e = 0; e < OCTET; ++e) x[u][e] = y[u][e] = 0.f;
            }
        }
        float t = 0.f;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            t += sum_of_products(x[u], METRIC ? y[u] : x[u]);
        }
        sum.add(t);
    }
    return sum;
}
// The same over the block, from values scaled by powers of two (unscaled where
// one is not finite).
template <int DT, int YT>
__device__ __noinline__ double scaled_sum(const ClipJob &j, long long lo, long long hi) {
    constexpr int Y = YT != NO_Y ? YT : DT;
    const char *yb = j.y ? j.y : j.x;
    const long long ld_y = j.y ? j.ld_y : j.ld;
    unsigned mx = 0, my = 0;
    float x[OCTET], y[OCTET];
    for (long long i = lo + threadIdx.x; i < hi; i += CLIP_THREADS) {
        const Place p = place_of(j, i);
        octet<DT>(j.x, j.ld, p, j.cols, false, x);
        octet<Y>(yb, ld_y, p, j.cols, false, y);
        for (int e = 0; e < OCTET; ++e) {
            mx = max(mx, __float_as_uint(x[e]) & 0x7fffffffu);
            my = max(my, __float_as_uint(y[e]) & 0x7fffffffu);
        }
    }
    mx = block_max(mx);
    my = block_max(my);
    const bool scale = mx < 0x7f800000u && my < 0x7f800000u;
    const int ex = scale ? to_one(mx) : 0, ey = scale ? to_one(my) : 0;
    const float fx = pow2(ex), fy = pow2(ey);
    Wide sum{};
    for (long long i = lo + threadIdx.x; i < hi; i += CLIP_THREADS) {
        const Place p = place_of(j, i);
        octet<DT>(j.x, j.ld, p, j.cols, false, x);
        octet<Y>(yb, ld_y, p, j.cols, false, y);
        for (int e = 0; e < OCTET; ++e) sum.add((x[e] * fx) * (y[e] * fy));
    }
    return ldexp(block_wide(sum).value(), -ex - ey);
}
template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, CLIP_PER_SM) clip_norm_kernel(const __grid_constant__ ClipParams<MAX> P) {
    pdl_wait();
    pdl_trigger();
    Wide mine{};
    for (long long lo = P.tile * blockIdx.x; lo < P.octets; lo += P.tile * gridDim.x) {
    const long long hi = min(P.octets, lo + P.tile);
    for (int n = job_of(P, lo); n < P.n && P.job[n].first < hi; ++n) {
        const ClipJob &j = P.job[n];
        const long long a = max(lo, j.first) - j.first, b = min(hi - j.first, j.rows * j.per_row);
        by_types(j, [&](auto t) { products<t.DT, t.YT>(j, n, a, b, mine); });
    }
    }
    // every warp joins the warps' sums, and hi is the same for all threads
    const Wide s = block_wide(mine);
    double sum = s.value();
    if (!finite(s.hi) || fabsf(s.hi) < 1e-28f) {
        sum = 0;
        for (long long lo = P.tile * blockIdx.x; lo < P.octets; lo += P.tile * gridDim.x) {
        const long long hi = min(P.octets, lo + P.tile);
        for (int n = job_of(P, lo); n < P.n && P.job[n].first < hi; ++n) {
            const ClipJob &j = P.job[n];
            const long long a = max(lo, j.first) - j.first, b = min(hi - j.first, j.rows * j.per_row);
            sum += by_types(j, [&](auto t) { return scaled_sum<t.DT, t.YT>(j, a, b); });
        }
        }
    }
    if (threadIdx.x == 0) P.part[P.part0 + blockIdx.x] = sum;
}

// N octets of a tensor without gaps: one at x (and out, w), the others each
// `back` octets before it.
template <int DT, bool W, bool ANY, int N>
__device__ __forceinline__ void apply_octets(const char *x, int ox, char *out, int out_dtype, float *w, float scale,
                                             float eta) {
    constexpr int ES = Elem<DT>::N == 4 ? 4 : 2, BACK = CLIP_THREADS * OCTET;
    const int es_out = out_dtype == KFAC_F32 ? 4 : 2;
    Raw<DT, ANY> r[N];
    float4 p[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        r[k].load(x - k * BACK * ES, ox);
        if (W) {
            const float4 *q = reinterpret_cast<const float4 *>(w - k * BACK);
            p[k][0] = q[0];
            p[k][1] = q[1];
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float v[OCTET];
        r[k].values(ox, v);
#pragma unroll
        for (int e = 0; e < OCTET; ++e) v[e] *= scale;
        if (out) {
            char *o = out - k * BACK * es_out;
            if (out_dtype == KFAC_BF16) store8<KFAC_BF16>(o, v);
            else if (out_dtype == KFAC_F16) store8<KFAC_F16>(o, v);
            else store8<KFAC_F32>(o, v);
        }
        if (W) {
            float4 *q = reinterpret_cast<float4 *>(w - k * BACK);
            q[0] = make_float4(p[k][0].x - eta * v[0], p[k][0].y - eta * v[1], p[k][0].z - eta * v[2],
                               p[k][0].w - eta * v[3]);
            q[1] = make_float4(p[k][1].x - eta * v[4], p[k][1].y - eta * v[5], p[k][1].z - eta * v[6],
                               p[k][1].w - eta * v[7]);
        }
    }
}
// The octets inside a tensor without gaps, from the end.
template <int DT, bool W, bool ANY>
__device__ __noinline__ void apply_inner(const ClipJob &j, long long a, long long b, float scale, float eta) {
    constexpr int ES = Elem<DT>::N == 4 ? 4 : 2, N = W ? 2 : 4;
    const int es_out = j.out_dtype == KFAC_F32 ? 4 : 2;
    long long left = b - a - threadIdx.x;             // octets up to this thread's
    const long long c = (a + left - 1) * OCTET - j.shift;  // its first element
    const char *x = j.x + c * ES;
    char *out = j.out ? j.out + c * es_out : nullptr;
    float *w = W ? j.w + c : nullptr;
    const int ox = (int)((uintptr_t)x & 15);
    auto back = [&](int n) {
        x -= (long long)n * CLIP_THREADS * OCTET * ES;
        if (out) out -= (long long)n * CLIP_THREADS * OCTET * es_out;
        if (W) w -= (long long)n * CLIP_THREADS * OCTET;
        left -= n * CLIP_THREADS;
    };
    for (; left > (N - 1) * CLIP_THREADS; back(N)) apply_octets<DT, W, ANY, N>(x, ox, out, j.out_dtype, w, scale, eta);
    for (; left > 0; back(1)) apply_octets<DT, W, ANY, 1>(x, ox, out, j.out_dtype, w, scale, eta);
}
template <int DT>
__device__ __noinline__ void apply_outer(const ClipJob &j, long long lo, long long hi, int tid, int nt, float scale,
                                         float eta);
// (short runs and ends as in the first pass)
template <int DT>
__device__ __forceinline__ void apply_run(const ClipJob &j, int n, long long lo, long long hi, float scale, float eta) {
    const int lane = threadIdx.x % 32;
    const bool mine = (int)threadIdx.x / 32 == n % (CLIP_THREADS / 32);
    if (hi - lo < SHORT_RUN) {
        if (mine) apply_outer<DT>(j, lo, hi, lane, 32, scale, eta);
        return;
    }
    long long a, b;
    inner_run(j, lo, hi, a, b);
    if (b > a && (!j.out || j.out_vec)) {
        if (mine) apply_outer<DT>(j, b, hi, lane, 32, scale, eta);
        if (mine) apply_outer<DT>(j, lo, a, lane, 32, scale, eta);
        const bool any = ((uintptr_t)j.x - (uintptr_t)j.shift * (Elem<DT>::N == 4 ? 4 : 2)) & 15;
        if (j.w) {
            if (any) apply_inner<DT, true, true>(j, a, b, scale, eta);
            else apply_inner<DT, true, false>(j, a, b, scale, eta);
        } else {
            if (any) apply_inner<DT, false, true>(j, a, b, scale, eta);
            else apply_inner<DT, false, false>(j, a, b, scale, eta);
        }
    } else {
        apply_outer<DT>(j, lo, hi, threadIdx.x, CLIP_THREADS, scale, eta);
    }
}
template <int DT>
__device__ __noinline__ void apply_outer(const ClipJob &j, long long lo, long long hi, int tid, int nt, float scale,
                                            float eta) {
    const int es_out = j.out_dtype == KFAC_F32 ? 4 : 2;
    // from the end of the run
    for (long long i = hi - 1 - tid; i >= lo; i -= nt) {
        const Place p = place_of(j, i);
        float x[OCTET];
        octet<DT>(j.x, j.ld, p, j.cols, j.vec, x);
#pragma unroll
        for (int e = 0; e < OCTET; ++e) x[e] *= scale;
        if (j.out) {
            char *row = j.out + p.row * j.ld_out * es_out;
            if (j.out_vec && p.whole) {
                char *at = row + p.col * es_out;
                if (j.out_dtype == KFAC_BF16) store8<KFAC_BF16>(at, x);
                else if (j.out_dtype == KFAC_F16) store8<KFAC_F16>(at, x);
                else store8<KFAC_F32>(at, x);
            } else {
#pragma unroll
                for (int e = 0; e < OCTET; ++e) {
                    const long long c = p.col + e;
                    if (c < 0 || c >= j.cols) continue;
                    if (j.out_dtype == KFAC_BF16) ((uint16_t *)row)[c] = Elem<KFAC_BF16>::round(x[e]);
                    else if (j.out_dtype == KFAC_F16) ((uint16_t *)row)[c] = Elem<KFAC_F16>::round(x[e]);
                    else ((float *)row)[c] = x[e];
                }
            }
        }
        if (j.w) {
            float *row = j.w + p.row * j.ld_w;
            if (j.vec && p.whole) {
                float4 *at = reinterpret_cast<float4 *>(row + p.col);
                float4 a = at[0], b = at[1];
                a.x -= eta * x[0]; a.y -= eta * x[1]; a.z -= eta * x[2]; a.w -= eta * x[3];
                b.x -= eta * x[4]; b.y -= eta * x[5]; b.z -= eta * x[6]; b.w -= eta * x[7];
                at[0] = a;
                at[1] = b;
            } else {
#pragma unroll
                for (int e = 0; e < OCTET; ++e)
                    if (p.col + e >= 0 && p.col + e < j.cols) row[p.col + e] -= eta * x[e];
            }
        }
    }
}

// norm and scale from the sum of products.
__device__ __forceinline__ float scale_of(double sum, float max_norm, float &norm) {
    norm = (float)sqrt(sum < 0 ? 0. : sum);
    return norm > max_norm ? max_norm / norm : norm <= max_norm ? 1.f : norm;
}

// Few small tensors in one launch: a cluster of CTAs takes the sum of products,
// joins it through shared memory, and applies the scale.  The sums are
// the only ones that cross CTAs, so that no CTA waits for memory that another writes.
constexpr int CLIP_CLUSTER = 8;
__global__ void __launch_bounds__(CLIP_THREADS) clip_small_kernel(const __grid_constant__ ClipParams<CLIP_FEW> P) {
    __shared__ double parts[CLIP_CLUSTER];
    cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const int rank = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x;
    const long long lo = P.octets * rank / ctas, hi = P.octets * (rank + 1) / ctas;
    Wide mine{};
    for (int n = 0; n < P.n; ++n) {
        const ClipJob &j = P.job[n];
        const long long a = max(lo, j.first) - j.first, b = min(hi - j.first, j.rows * j.per_row);
        if (b <= a) continue;
        mine = by_types(j, [&](auto t) { return outer_products<t.DT, t.YT>(j, a, b, tid, CLIP_THREADS, mine); });
    }
    const Wide s = block_wide(mine);
    double sum = s.value();
    if (!finite(s.hi) || fabsf(s.hi) < 1e-28f) {
        sum = 0;
        for (int n = 0; n < P.n; ++n) {
            const ClipJob &j = P.job[n];
            const long long a = max(lo, j.first) - j.first, b = min(hi - j.first, j.rows * j.per_row);
            if (b <= a) continue;
            sum += by_types(j, [&](auto t) { return scaled_sum<t.DT, t.YT>(j, a, b); });
        }
    }
    cluster_wait();
    if (tid == 0)
        for (int c = 0; c < ctas; ++c) {
            double *there;
            asm volatile("mapa.u64 %0, %1, %2;" : "=l"(there) : "l"(&parts[rank]), "r"(c));
            *there = sum;
        }
    cluster_sync();
    double all = 0;
    for (int c = 0; c < ctas; ++c) all += parts[c];
    float norm;
    const float scale = scale_of(all, P.max_norm, norm);
    if (rank == 0 && tid == 0) {
        if (P.norm) *P.norm = norm;
        if (P.scale) *P.scale = scale;
        *P.err = finite(norm) ? 0 : ERR_NONFINITE;
    }
    for (int n = 0; n < P.n; ++n) {
        const ClipJob &j = P.job[n];
        const long long a = max(lo, j.first) - j.first, b = min(hi - j.first, j.rows * j.per_row);
        if (b <= a || (!j.w && (!j.out || (j.out == j.x && scale == 1.f)))) continue;
        if (j.dtype == KFAC_BF16) apply_outer<KFAC_BF16>(j, a, b, tid, CLIP_THREADS, scale, P.eta);
        else if (j.dtype == KFAC_F16) apply_outer<KFAC_F16>(j, a, b, tid, CLIP_THREADS, scale, P.eta);
        else apply_outer<KFAC_F32>(j, a, b, tid, CLIP_THREADS, scale, P.eta);
    }
}

// Every CTA adds up the first pass's sums itself (the same sum in the same order).
template <int MAX>
__global__ void __launch_bounds__(CLIP_THREADS, CLIP_PER_SM) clip_apply_kernel(const __grid_constant__ ClipParams<MAX> P) {
    __shared__ float shared_scale;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < 32) {
        double s = 0;
        for (int i = threadIdx.x; i < P.parts; i += 32) s += P.part[i];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_down_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            float norm;
            const float scale = scale_of(s, P.max_norm, norm);
            shared_scale = scale;
            if (blockIdx.x == 0 && P.err) {
                if (P.norm) *P.norm = norm;
                if (P.scale) *P.scale = scale;
                *P.err = finite(norm) ? 0 : ERR_NONFINITE;
            }
        }
    }
    __syncthreads();
    const float scale = shared_scale;
    const long long tiles = (P.octets + P.tile - 1) / P.tile;
    for (long long t = tiles - 1 - blockIdx.x; t >= 0; t -= gridDim.x) {
    const long long lo = t * P.tile, hi = min(P.octets, lo + P.tile);
    for (int n = job_of(P, hi - 1); n >= 0 && P.job[n].first + P.job[n].rows * P.job[n].per_row > lo; --n) {
        const ClipJob &j = P.job[n];
        if (!j.w && (!j.out || (j.out == j.x && scale == 1.f))) continue;
        const long long a = max(lo, j.first) - j.first, b = min(hi - j.first, j.rows * j.per_row);
        if (j.dtype == KFAC_BF16) apply_run<KFAC_BF16>(j, n, a, b, scale, P.eta);
        else if (j.dtype == KFAC_F16) apply_run<KFAC_F16>(j, n, a, b, scale, P.eta);
        else apply_run<KFAC_F32>(j, n, a, b, scale, P.eta);
    }
    }
}

bool known(int dtype) { return dtype == KFAC_BF16 || dtype == KFAC_F16 || dtype == KFAC_F32; }
int size_of(int dtype) { return dtype == KFAC_F32 ? 4 : 2; }

kfac_status check_clip(const kfac_clip_desc *descs, int count, float max_norm, float eta) {
    if (count < 0 || (count > 0 && !descs) || !(max_norm > 0.f) || !std::isfinite(eta)) return KFAC_ERR_INVALID;
    for (int i = 0; i < count; ++i) {
        const kfac_clip_desc &d = descs[i];
        if (d.rows < 0 || d.cols < 0 || !known(d.dtype) || (d.out && !known(d.out_dtype)) || (d.y && !known(d.y_dtype)))
            return KFAC_ERR_INVALID;
        if (d.y && d.y_dtype != d.dtype && d.dtype != KFAC_F32) return KFAC_ERR_INVALID;
        if (d.rows == 0 || d.cols == 0) continue;
        if (!d.x || d.ld < d.cols || (d.y && d.ld_y < d.cols) || (d.out && d.ld_out < d.cols) ||
            (d.w && d.ld_w < d.cols))
            return KFAC_ERR_INVALID;
        if ((uintptr_t)d.x % size_of(d.dtype) || (d.y && (uintptr_t)d.y % size_of(d.y_dtype)) ||
            (d.out && (uintptr_t)d.out % size_of(d.out_dtype)) || (uintptr_t)d.w % 4)
            return KFAC_ERR_INVALID;
        if (d.out == d.x && (d.out_dtype != d.dtype || d.ld_out != d.ld)) return KFAC_ERR_INVALID;
    }
    return KFAC_OK;
}

ClipJob job_from(const kfac_clip_desc &d, bool apply) {
    ClipJob j{(const char *)d.x, (const char *)d.y, (char *)d.out, d.w, d.ld, d.ld_y, d.ld_out, d.ld_w,
              d.rows, d.cols, 0, 0, (uint8_t)d.dtype, (uint8_t)d.y_dtype, (uint8_t)d.out_dtype, 0, 0, 0};
    if (d.rows == 1 || (d.ld == d.cols && (!d.y || d.ld_y == d.cols) && (!d.out || d.ld_out == d.cols) &&
                        (!d.w || d.ld_w == d.cols))) {
        j.cols = d.rows * d.cols;
        j.rows = 1;
    }
    // The octets lie so that x is taken on 16-byte boundaries in the first pass, and
    // w, else out, in the second; what is only read may lie anywhere.  What is read
    // and written has to be on the boundaries.
    const int es = size_of(d.dtype), es_out = size_of(d.out_dtype);
    const uintptr_t lead = !apply ? (uintptr_t)d.x : d.w ? (uintptr_t)d.w : (uintptr_t)d.out;
    const int es_lead = !apply ? es : d.w ? 4 : es_out;
    // rows that start alike modulo 16 bytes: ld a multiple of 8 elements, or one row
    const bool alike = j.rows == 1 || (d.ld % OCTET == 0 && (!d.y || d.ld_y % OCTET == 0) &&
                                       (!d.out || d.ld_out % OCTET == 0) && (!d.w || d.ld_w % OCTET == 0));
    if (alike) {
        j.shift = (uint8_t)((lead & 15) / es_lead);
        const auto aligned = [&](const void *p, int size) { return ((uintptr_t)p - (uintptr_t)j.shift * size) % 16 == 0; };
        j.out_vec = d.out && aligned(d.out, es_out);
        j.vec = !apply || d.out != d.x || j.out_vec;
    }
    j.per_row = ceil_div(j.cols + j.shift, OCTET);
    return j;
}

struct ClipPlan {
    int *err;
    double *part;
    int parts;
};
// CTAs of a launch over `octets`.  (144 tensors of 17 or 306 values, with metric and
// weights, take 14 us of the GPU's time; with 256 octets to a CTA at least, 24.)
int ctas_of(long long octets) {
    return (int)std::max<long long>(1, std::min<long long>(device_sm_count() * CLIP_PER_SM, ceil_div(octets, CTA_OCTETS)));
}
int tensors_of(int count) { return count <= CLIP_FEW ? CLIP_FEW : CLIP_MANY; }
ClipPlan plan_clip(int count, Arena &ws) {
    ClipPlan p;
    p.err = ws.take<int>(64);
    // (at most; a launch of few octets has fewer CTAs)
    p.parts = (int)std::max<long long>(1, ceil_div(count, tensors_of(count))) * device_sm_count() * CLIP_PER_SM;
    p.part = ws.take<double>((size_t)p.parts);
    return p;
}

// Both passes, in launches of MAX tensors.
template <int MAX>
kfac_status run_clip(const kfac_clip_desc *descs, int count, float max_norm, float eta, float *norm, float *scale,
                     const ClipPlan &plan, cudaStream_t st) {
    std::unique_ptr<ClipParams<MAX>> P(new ClipParams<MAX>);
    P->part = plan.part;
    P->max_norm = max_norm;
    P->eta = eta;
    P->norm = norm;
    P->scale = scale;
    const int launches = std::max(1, (count + MAX - 1) / MAX);
    auto fill = [&](int launch, bool apply) {
        P->n = 0;
        P->octets = 0;
        for (int i = launch * MAX; i < std::min(count, launch * MAX + MAX); ++i) {
            if (descs[i].rows == 0 || descs[i].cols == 0) continue;
            ClipJob j = job_from(descs[i], apply);
            j.first = P->octets;
            P->octets += (long long)align_up((size_t)(j.rows * j.per_row), LINE);
            P->job[P->n++] = j;
        }
        P->tile = std::max<long long>(1, ceil_div(P->octets, ctas_of(P->octets)));
        // In the first pass tiles of about TILE octets, the same number for every CTA.  Tiles
        // and tensors begin on memory's lines: 1.0e9 bf16 values take 973 us, 1007 where they
        // begin anywhere.
        long long unit = apply ? 64 : 512;
        while (unit > LINE && unit * 8 > P->tile) unit /= 2;
        P->tile = (long long)align_up((size_t)(apply ? P->tile : ceil_div(P->tile, ceil_div(P->tile, TILE))), unit);
    };
    if constexpr (MAX == CLIP_FEW) {
        fill(0, true);
        // (six tensors of 9 k octets take 26 us in two launches and 19 in one cluster's, six of
        // 40 k octets 22 and 31)
        if (P->octets <= SMALL_OCTETS) {
            P->err = plan.err;
            unsigned ctas = 1;
            while (ctas < CLIP_CLUSTER && (long long)ctas * CLIP_THREADS * 2 < P->octets) ctas *= 2;
            KFAC_LAUNCH_CLUSTERS(KK_CLIP_NORM, st, clip_small_kernel, ctas, ctas, CLIP_THREADS, 0, *P);
            return KFAC_OK;
        }
    }
    int parts = 0;
    for (int l = 0; l < launches; ++l) {
        fill(l, false);
        P->part0 = parts;
        if (P->n == 0) continue;
        const int ctas = ctas_of(P->octets);
        parts += ctas;
        KFAC_LAUNCH(KK_CLIP_NORM, st, (clip_norm_kernel<MAX>), ctas, CLIP_THREADS, 0, *P);
    }
    P->parts = parts;
    for (int l = 0; l < launches; ++l) {
        fill(l, true);
        bool writes = false;
        for (int i = 0; i < P->n; ++i) writes |= P->job[i].out || P->job[i].w;
        if (l > 0 && !writes) continue;
        P->err = l == 0 ? plan.err : nullptr;
        if (!writes) P->octets = 0;
        KFAC_LAUNCH(KK_CLIP_APPLY, st, (clip_apply_kernel<MAX>), writes ? ctas_of(P->octets) : 1, CLIP_THREADS, 0, *P);
    }
    return KFAC_OK;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" size_t kfac_clip_norm_workspace_size(const kfac_clip_desc *descs, int count) {
    if (check_clip(descs, count, 1.f, 0.f) != KFAC_OK) return 0;
    Arena a;
    plan_clip(count, a);
    return a.used;
}

extern "C" kfac_status kfac_clip_norm(const kfac_clip_desc *descs, int count, float max_norm, float eta, float *norm,
                                      float *scale, void *workspace, size_t workspace_bytes, void *stream) {
    kfac_status s = check_clip(descs, count, max_norm, eta);
    if (s != KFAC_OK) return s;
    if (!workspace || ((uintptr_t)workspace % 256) != 0) return KFAC_ERR_WORKSPACE;
    Arena ws(workspace, workspace_bytes);
    const ClipPlan plan = plan_clip(count, ws);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    DeviceMemory memory;
    for (int i = 0; i < count; ++i) {
        const kfac_clip_desc &d = descs[i];
        if (!memory.holds(d.x, 0) || !memory.holds(d.y, 1) || !memory.holds(d.out, 2) || !memory.holds(d.w, 3))
            return KFAC_ERR_INVALID;
    }
    if (!all_on_this_device({norm, scale})) return KFAC_ERR_INVALID;
    cudaStream_t st = (cudaStream_t)stream;
    return count <= CLIP_FEW ? run_clip<CLIP_FEW>(descs, count, max_norm, eta, norm, scale, plan, st)
                             : run_clip<CLIP_MANY>(descs, count, max_norm, eta, norm, scale, plan, st);
}
