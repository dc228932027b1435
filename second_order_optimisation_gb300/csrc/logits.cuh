// logits.cuh -- device helpers of the losses on logits: 16-byte groups of a
// row that may start at any element, and the running statistics of a softmax.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.h"

namespace kfac {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float F32_MAX = 3.402823466e38f;
// Exponents (base 2) are cut off here where they are multiplied with their own
// power of two: 2^-10000 is 0 in fp32, and 0 * -10000 is 0 where 0 * -inf is not.
constexpr float Y_FLOOR = -1e4f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= F32_MAX; }

// Two fp32 values in one 64-bit register pair: one instruction for both.
struct f2 {
    unsigned long long v;
};
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both(f2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ f2 add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ f2 ex2(f2 a) {
    const float2 x = both(a);
    return pair(ex2(x.x), ex2(x.y));
}
__device__ __forceinline__ f2 max2(f2 a, float b) {
    const float2 x = both(a);
    return pair(fmaxf(x.x, b), fmaxf(x.y, b));
}

// A sum of many terms that may differ by more than fp32's 24 bits: s + c, c the
// bits that the additions to s have lost (a row's most likely token gives a
// term of 1; without c, thousands of terms near 2^-25 would vanish beside it).
struct Sum2 {
    f2 s, c;
    __device__ __forceinline__ Sum2() : s(pair(0.f, 0.f)), c(s) {}
    __device__ __forceinline__ void add(f2 b) {
        const f2 m1 = pair(-1.f, -1.f);
        const f2 t = kfac::add(s, b), bb = fma(s, m1, t);                 // bb = t - s
        const f2 ds = fma(fma(bb, m1, t), m1, s), db = fma(bb, m1, b);    // s - (t - bb), b - bb
        c = kfac::add(c, kfac::add(ds, db));
        s = t;
    }
    __device__ __forceinline__ float total() const {
        const float2 a = both(s), b = both(c);
        return (a.x + a.y) + (b.x + b.y);
    }
};

// A sum kept as hi + lo (about 45 bits): fp64 additions are too slow here to be
// made by every thread.
struct Wide {
    float hi, lo;
    __device__ __forceinline__ void add(float b) {
        const float t = __fadd_rn(hi, b), bb = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, bb)), __fsub_rn(b, bb)));
        hi = t;
    }
    __device__ __forceinline__ void add(Wide b) {
        add(b.hi);
        lo = __fadd_rn(lo, b.lo);
    }
    __device__ __forceinline__ Wide shuffled(int o) const {
        Wide r;
        r.hi = __shfl_xor_sync(0xffffffffu, hi, o);
        r.lo = __shfl_xor_sync(0xffffffffu, lo, o);
        return r;
    }
    // Over the lanes of a warp; lane 0's is the one to take.
    __device__ __forceinline__ void add_lanes() {
        for (int o = 16; o > 0; o >>= 1) add(shuffled(o));
    }
    // An overflow to infinity leaves hi at it and NaN in lo.
    __device__ __forceinline__ double value() const { return finite(hi) ? (double)hi + (double)lo : (double)hi; }
};

// A 16-byte group of elements of one type, as bits and as fp32 values.
template <int DT>
struct Elem;
template <>
struct Elem<KFAC_F32> {
    using bits = uint32_t;
    static constexpr int N = 4;
    static constexpr uint32_t NEG_INF = 0xff800000u;  // -inf in every element of a 32-bit word
    static __device__ __forceinline__ float value(bits b) { return __uint_as_float(b); }
    using two = f2;  // running maximum of groups (NaN is passed over)
    static __device__ __forceinline__ two lowest() { return pair(-F32_MAX, -F32_MAX); }
    static __device__ __forceinline__ two nothing() { return pair(-INFINITY, -INFINITY); }
    static __device__ __forceinline__ two raise(two m, uint4 u) {
        const float2 a = both(m);
        return pair(fmaxf(a.x, fmaxf(__uint_as_float(u.x), __uint_as_float(u.y))),
                    fmaxf(a.y, fmaxf(__uint_as_float(u.z), __uint_as_float(u.w))));
    }
    static __device__ __forceinline__ float largest(two m) {
        const float2 a = both(m);
        return fmaxf(a.x, a.y);
    }
    static __device__ __forceinline__ uint32_t bounded1(uint32_t v) {
        asm("max.NaN.f32 %0, %0, 0fF0000000;" : "+r"(v));  // BOUND
        return v;
    }
    static constexpr float BOUND = -0x1p97f;  // -1.6e29
    static __device__ __forceinline__ uint4 bounded(uint4 u) {
        return make_uint4(bounded1(u.x), bounded1(u.y), bounded1(u.z), bounded1(u.w));
    }
    static __device__ __forceinline__ bits round(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ void unpack(uint4 u, float *v) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};
template <>
struct Elem<KFAC_BF16> {
    using bits = uint16_t;
    static constexpr int N = 8;
    static constexpr uint32_t NEG_INF = 0xff80ff80u;
    static __device__ __forceinline__ float value(bits b) { return __uint_as_float((uint32_t)b << 16); }
    using two = __nv_bfloat162;  // running maximum of groups (NaN is passed over)
    static __device__ __forceinline__ two as_two(uint32_t w) { return *reinterpret_cast<two *>(&w); }
    static __device__ __forceinline__ two lowest() { return as_two(0xff7fff7fu); }
    static __device__ __forceinline__ two nothing() { return as_two(NEG_INF); }
    static __device__ __forceinline__ uint32_t bounded1(uint32_t v) {
        const two b = __hmax2_nan(as_two(v), as_two(0xf000f000u));  // BOUND
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    static constexpr float BOUND = -0x1p97f;  // -1.6e29
    static __device__ __forceinline__ uint4 bounded(uint4 u) {
        return make_uint4(bounded1(u.x), bounded1(u.y), bounded1(u.z), bounded1(u.w));
    }
    static __device__ __forceinline__ two raise(two m, uint4 u) {
        return __hmax2(m, __hmax2(__hmax2(as_two(u.x), as_two(u.y)), __hmax2(as_two(u.z), as_two(u.w))));
    }
    static __device__ __forceinline__ float largest(two m) { return fmaxf(__low2float(m), __high2float(m)); }
    static __device__ __forceinline__ bits round(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
    static __device__ __forceinline__ void unpack2(uint32_t u, float *v) {
        v[0] = __uint_as_float(u << 16);
        v[1] = __uint_as_float(u & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack2(const float *v) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    static __device__ __forceinline__ void unpack(uint4 u, float *v) {
        unpack2(u.x, v); unpack2(u.y, v + 2); unpack2(u.z, v + 4); unpack2(u.w, v + 6);
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        return make_uint4(pack2(v), pack2(v + 2), pack2(v + 4), pack2(v + 6));
    }
};
template <>
struct Elem<KFAC_F16> {
    using bits = uint16_t;
    static constexpr int N = 8;
    static constexpr uint32_t NEG_INF = 0xfc00fc00u;
    static __device__ __forceinline__ float value(bits b) { return __half2float(__ushort_as_half(b)); }
    using two = __half2;  // running maximum of groups (NaN is passed over)
    static __device__ __forceinline__ two as_two(uint32_t w) { return *reinterpret_cast<two *>(&w); }
    static __device__ __forceinline__ two lowest() { return as_two(0xfbfffbffu); }
    static __device__ __forceinline__ two nothing() { return as_two(NEG_INF); }
    static __device__ __forceinline__ uint32_t bounded1(uint32_t v) {
        const two b = __hmax2_nan(as_two(v), as_two(0xfbfffbffu));  // BOUND
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    static constexpr float BOUND = -65504.f;  // the lowest finite value
    static __device__ __forceinline__ uint4 bounded(uint4 u) {
        return make_uint4(bounded1(u.x), bounded1(u.y), bounded1(u.z), bounded1(u.w));
    }
    static __device__ __forceinline__ two raise(two m, uint4 u) {
        return __hmax2(m, __hmax2(__hmax2(as_two(u.x), as_two(u.y)), __hmax2(as_two(u.z), as_two(u.w))));
    }
    static __device__ __forceinline__ float largest(two m) { return fmaxf(__low2float(m), __high2float(m)); }
    static __device__ __forceinline__ bits round(float v) { return __half_as_ushort(__float2half_rn(v)); }
    static __device__ __forceinline__ void unpack2(uint32_t u, float *v) {
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&u));
        v[0] = f.x;
        v[1] = f.y;
    }
    static __device__ __forceinline__ uint32_t pack2(const float *v) {
        __half2 h = __floats2half2_rn(v[0], v[1]);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    static __device__ __forceinline__ void unpack(uint4 u, float *v) {
        unpack2(u.x, v); unpack2(u.y, v + 2); unpack2(u.z, v + 4); unpack2(u.w, v + 6);
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        return make_uint4(pack2(v), pack2(v + 2), pack2(v + 4), pack2(v + 6));
    }
};

__device__ __forceinline__ uint4 ld16(const char *p) { return *reinterpret_cast<const uint4 *>(p); }

// Q times 16 bytes from any element boundary, by aligned loads.  ANY: `off` is the
// address modulo 16, not 0 and the same for all threads, and the pieces that the
// bytes lie in reach less than 16 bytes before and behind them.
template <int Q, bool ANY>
struct Pieces {
    uint4 u[Q + ANY];
    __device__ __forceinline__ void load(const char *p, int off) {
#pragma unroll
        for (int q = 0; q < Q + ANY; ++q) u[q] = ld16(ANY ? p - off + 16 * q : p + 16 * q);
    }
    __device__ __forceinline__ void take(int off, uint4 *v) const {
        if constexpr (!ANY) {
#pragma unroll
            for (int q = 0; q < Q; ++q) v[q] = u[q];
        } else {
            shift(off, v);
        }
    }
    __device__ __forceinline__ void shift(int off, uint4 *v) const {
        uint32_t w[4 * (Q + 1)];
#pragma unroll
        for (int q = 0; q <= Q; ++q) w[4 * q] = u[q].x, w[4 * q + 1] = u[q].y, w[4 * q + 2] = u[q].z, w[4 * q + 3] = u[q].w;
        // left by 8, 4 and 2 bytes as the offset has them
        if (off & 8)
#pragma unroll
            for (int i = 0; i + 2 < 4 * (Q + 1); ++i) w[i] = w[i + 2];
        if (off & 4)
#pragma unroll
            for (int i = 0; i + 1 < 4 * (Q + 1); ++i) w[i] = w[i + 1];
        if (off & 2)
#pragma unroll
            for (int i = 0; i + 1 < 4 * (Q + 1); ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
#pragma unroll
        for (int q = 0; q < Q; ++q) v[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
};

// A row of `n` elements that may start anywhere: group g holds the elements
// g N - phase .. g N - phase + N - 1 that exist, and starts on a 16-byte boundary.
template <int DT>
struct Row {
    using E = Elem<DT>;
    using bits = typename E::bits;
    const char *base;  // 16-byte boundary at or before the first element
    int phase, n;
    __device__ __forceinline__ Row(const void *p, int n_) : n(n_) {
        const uintptr_t a = (uintptr_t)p;
        phase = (int)(a & 15) / (int)sizeof(bits);
        base = (const char *)(a & ~(uintptr_t)15);
    }
    __device__ __forceinline__ int groups() const { return (phase + n + E::N - 1) / E::N; }
    __device__ __forceinline__ int first(int g) const { return g * E::N - phase; }
    // Whole groups are begin() .. end() - 1; the elements of group 0 before them
    // (where phase > 0) and those of group end() behind them are the edges.
    __device__ __forceinline__ int begin() const { return phase > 0; }
    __device__ __forceinline__ int end() const { return max((phase + n) / E::N, begin()); }
    __device__ __forceinline__ bool has_front() const { return phase > 0; }
    __device__ __forceinline__ bool has_back() const { return end() * E::N < phase + n; }
    __device__ __forceinline__ uint4 load_whole(int g) const {
        uint4 u;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(base + (size_t)g * 16)
                     : "memory");
        return u;
    }
    static __device__ __forceinline__ uint4 none() { return make_uint4(E::NEG_INF, E::NEG_INF, E::NEG_INF, E::NEG_INF); }
    // An edge group's bits, -inf where there is no element.
    __device__ __forceinline__ uint4 load_edge(int g) const { return edge_group(base + (size_t)g * 16, first(g), n); }
    static __device__ __noinline__ uint4 edge_group(const char *at, int e0, int n) {
        const bits *p = reinterpret_cast<const bits *>(at);
        uint32_t w[4] = {E::NEG_INF, E::NEG_INF, E::NEG_INF, E::NEG_INF};
#pragma unroll
        for (int i = 0; i < E::N; ++i) {
            if (e0 + i < 0 || e0 + i >= n) continue;
            const uint32_t b = p[i];
            if (E::N == 4)
                w[i] = b;
            else
                w[i / 2] = (i & 1) ? ((w[i / 2] & 0xffffu) | (b << 16)) : ((w[i / 2] & 0xffff0000u) | b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Writes an edge group's elements to the row at `out`.
    static __device__ __noinline__ void store_edge(void *out, int e0, int n, uint4 u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < E::N; ++i)
            if (e0 + i >= 0 && e0 + i < n) ((bits *)out)[e0 + i] = (bits)(E::N == 4 ? w[i] : w[i / 2] >> (i & 1) * 16);
    }
};

// Statistics of a part of a row: m its maximum (at least the lowest finite
// value, so that z = -inf gives 2^-inf = 0), s = sum_j 2^y_j and (ENT) t =
// sum_j 2^y_j y_j with y_j = (z_j - m) k.  A NaN or +inf makes s NaN.
struct Part {
    float m, s, t;
};

// Lanes' maximum, the same on each of `width` lanes (`mask`: the lanes that come
// here together).
constexpr unsigned ALL_LANES = 0xffffffffu;
__device__ __forceinline__ float lanes_max(float v, int width, unsigned mask = ALL_LANES) {
    for (int o = width / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
    return v;
}
__device__ __forceinline__ float lanes_sum(float v, int width, unsigned mask = ALL_LANES) {
    for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

// A group's values as pairs.
template <int DT>
__device__ __forceinline__ void unpack_pairs(uint4 u, f2 *v) {
    float f[Elem<DT>::N];
    Elem<DT>::unpack(u, f);
#pragma unroll
    for (int i = 0; i < Elem<DT>::N / 2; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}

// (z - m) k in one multiply-add, z k - c with c = m k rounded: exact but for the
// result's own rounding, and for delta = m k - c, which is the same for the whole
// row and is put back into the sums (2^y (z) = 2^-delta 2^(z k - c)).  `ok` is false
// where m k is so large that c or delta would be (rows at the type's lowest value):
// then the difference is formed before the product.
struct Shift {
    float m, k, c, delta;
    bool ok;
    __device__ __forceinline__ Shift(float m_, float k_, bool allowed) : m(m_), k(k_), c(m_ * k_) {
        ok = allowed && fabsf(c) < 1048576.f;
        delta = ok ? fmaf(m, k, -c) : 0.f;
    }
    template <bool FAST>
    __device__ __forceinline__ f2 apply(f2 z) const {
        return FAST ? fma(z, pair(k, k), pair(-c, -c)) : mul(add(z, pair(-m, -m)), pair(k, k));
    }
};

// With an entropy the fast form multiplies 2^y with y (and, in a gradient, with a factor
// b), and logits of -inf are raised to Elem::BOUND first, so that 0 is not multiplied with
// -inf.  That needs 2^y = 0 at the bound (y below -150: not so where the temperature, or
// the row's maximum, is near the bound's size) and a finite b y there (not so for a very
// small temperature); elsewhere the other form bounds y itself.
template <int DT, bool ENT>
__device__ __forceinline__ Shift shift_of(float m, float k, float b = 0.f) {
    const float far = (m - Elem<DT>::BOUND) * k;
    return Shift(m, k, !ENT || (far > 200.f && far * fmaxf(1.f, fabsf(b)) < 1e37f));
}

// Sums over groups whose maximum is at most the shift's.  A thread adds few
// groups, each summed as a tree first; a long run of groups takes Sum2's way.
template <int DT, bool ENT>
struct Sums {
    f2 s, t;
    __device__ __forceinline__ Sums() : s(pair(0.f, 0.f)), t(s) {}
    // (in the FAST form a logit at the bound or below has 2^y = 0, and its y must stay finite: shift_of)
    template <bool FAST>
    __device__ __forceinline__ f2 group(uint4 u, const Shift &h) {
        constexpr int H = Elem<DT>::N / 2;
        f2 v[H];
        unpack_pairs<DT>(ENT && FAST ? Elem<DT>::bounded(u) : u, v);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const f2 y = h.apply<FAST>(v[i]);
            v[i] = ex2(y);
            if (ENT) t = fma(v[i], FAST ? y : max2(y, Y_FLOOR), t);
        }
        if constexpr (H == 4) return kfac::add(kfac::add(v[0], v[1]), kfac::add(v[2], v[3]));
        else return kfac::add(v[0], v[1]);
    }
    template <bool FAST>
    __device__ __forceinline__ void add(uint4 u, const Shift &h) {
        s = kfac::add(s, group<FAST>(u, h));
    }
    __device__ __forceinline__ Part part(const Shift &h, int width) const {
        const float2 ss = both(s), tt = both(t);
        Part p{h.m, lanes_sum(ss.x + ss.y, width), ENT ? lanes_sum(tt.x + tt.y, width) : 0.f};
        const float c = ex2(-h.delta);
        if (ENT) p.t = c * fmaf(-h.delta, p.s, p.t);
        p.s *= c;
        return p;
    }
};

// A thread's statistics of many groups, taken in batches: its maximum rises as
// it goes, and the sums so far are scaled down with it.
template <int DT, bool ENT>
struct Running {
    Sum2 s;
    f2 t;
    float m, k;
    __device__ __forceinline__ explicit Running(float k_) : t(pair(0.f, 0.f)), m(-F32_MAX), k(k_) {}
    __device__ __forceinline__ void raise(float to) {
        if (to > m) {
            const float d = (m - to) * k, c = ex2(d), f = fmaxf(d, Y_FLOOR);
            const f2 c2 = pair(c, c);
            if (ENT) t = mul(c2, fma(pair(f, f), s.s, t));
            s.s = mul(s.s, c2);
            s.c = mul(s.c, c2);
            m = to;
        }
    }
    // `count` groups, the i-th to be passed over where the i-th bit of `skip` is set.
    template <int VPT>
    __device__ __forceinline__ void add(const uint4 *u, int count, unsigned skip) {
        auto best = Elem<DT>::lowest();
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i < count) best = Elem<DT>::raise(best, u[i]);
        raise(Elem<DT>::largest(best));
        const Shift h = shift_of<DT, ENT>(m, k);
        Sums<DT, ENT> batch;
        if (h.ok) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (i < count && !(skip >> i & 1)) batch.template add<true>(u[i], h);
        } else {
#pragma unroll 1
            for (int i = 0; i < VPT; ++i) {
                uint4 v = u[0];
#pragma unroll
                for (int q = 1; q < VPT; ++q) v = q == i ? u[q] : v;  // (registers have no index)
                if (i < count && !(skip >> i & 1)) batch.template add<false>(v, h);
            }
        }
        const float f = ex2(-h.delta);
        if (ENT) t = kfac::add(t, mul(pair(f, f), fma(pair(-h.delta, -h.delta), batch.s, batch.t)));
        s.add(mul(pair(f, f), batch.s));
    }
    // Of `width` lanes.
    __device__ __forceinline__ Part part(int width = 32, unsigned mask = ALL_LANES) {
        raise(lanes_max(m, width, mask));
        const float2 tt = both(t);
        return Part{m, lanes_sum(s.total(), width, mask), ENT ? lanes_sum(tt.x + tt.y, width, mask) : 0.f};
    }
};

// A part's sums, relative to a maximum M >= p.m.
template <bool ENT>
__device__ __forceinline__ Part relative_to(Part p, float M, float k) {
    const float d = (p.m - M) * k, c = ex2(d);
    // an empty part is 0 whatever d is
    return p.s == 0.f ? Part{M, 0.f, 0.f} : Part{M, p.s * c, ENT ? c * (p.t + fmaxf(d, Y_FLOOR) * p.s) : 0.f};
}

}  // namespace kfac
