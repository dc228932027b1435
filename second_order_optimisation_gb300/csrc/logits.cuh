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

// A 16-byte group of elements of one type, as bits and as fp32 values.
template <int DT>
struct Elem;
template <>
struct Elem<KFAC_F32> {
    using bits = uint32_t;
    static constexpr int N = 4;
    static constexpr uint32_t NEG_INF = 0xff800000u;  // -inf in every element of a 32-bit word
    static __device__ __forceinline__ float value(bits b) { return __uint_as_float(b); }
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
    __device__ __forceinline__ bool whole(int g) const { return first(g) >= 0 && first(g) + E::N <= n; }
    // The group's bits, -inf where there is no element.
    __device__ __forceinline__ uint4 load(int g) const {
        const char *p = base + (size_t)g * 16;
        uint4 u;
        if (whole(g)) {
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "l"(p)
                         : "memory");
            return u;
        }
        uint32_t w[4] = {E::NEG_INF, E::NEG_INF, E::NEG_INF, E::NEG_INF};
        const int e0 = first(g);
#pragma unroll
        for (int i = 0; i < E::N; ++i) {
            if (e0 + i < 0 || e0 + i >= n) continue;
            const uint32_t b = reinterpret_cast<const bits *>(p)[i];
            if (E::N == 4)
                w[i] = b;
            else
                w[i / 2] = (i & 1) ? ((w[i / 2] & 0xffffu) | (b << 16)) : ((w[i / 2] & 0xffff0000u) | b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Writes the group's values (element first(g) + i at v[i]) to the row at `out`.
template <int DT>
__device__ __forceinline__ void store_group(const Row<DT> &r, int g, void *out, bool same_phase, const float *v) {
    using E = Elem<DT>;
    typename E::bits *o = (typename E::bits *)out + r.first(g);
    if (same_phase && r.whole(g)) {
        *reinterpret_cast<uint4 *>(o) = E::pack(v);
        return;
    }
    const int e0 = r.first(g);
#pragma unroll
    for (int i = 0; i < E::N; ++i)
        if (e0 + i >= 0 && e0 + i < r.n) o[i] = E::round(v[i]);
}

// Running statistics of sum_j 2^((z_j - m) k): the maximum m, the sum s, and
// (ENT) t = sum_j 2^y y with y = (z_j - m) k.  m starts at the lowest finite
// value, so that z = -inf gives 2^-inf = 0; a NaN or +inf makes s NaN.
template <bool ENT>
struct Stat {
    float m, s, t;
    __device__ __forceinline__ Stat() : m(-F32_MAX), s(0.f), t(0.f) {}
    __device__ __forceinline__ void raise(float mx, float k) {
        if (mx > m) {
            const float d = (m - mx) * k, c = ex2(d);
            if (s != 0.f) {  // (a NaN sum stays)
                if (ENT) t = c * (t + fmaxf(d, Y_FLOOR) * s);
                s *= c;
            }
            m = mx;
        }
    }
    template <int N>
    __device__ __forceinline__ void add(const float *z, float k) {
        float mx = z[0];
#pragma unroll
        for (int i = 1; i < N; ++i) mx = fmaxf(mx, z[i]);
        raise(mx, k);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = (z[i] - m) * k, e = ex2(y);
            s += e;
            if (ENT) t = fmaf(e, fmaxf(y, Y_FLOOR), t);
        }
    }
    __device__ __forceinline__ void merge(float m2, float s2, float t2, float k) {
        if (m2 > m) {
            raise(m2, k);
            s += s2;
            if (ENT) t += t2;
        } else if (s2 != 0.f) {
            const float d = (m2 - m) * k, c = ex2(d);
            if (ENT) t += c * (t2 + fmaxf(d, Y_FLOOR) * s2);
            s = fmaf(s2, c, s);
        }
    }
    __device__ __forceinline__ void merge_lanes(float k, int width = 32) {
        for (int o = width / 2; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
            const float t2 = ENT ? __shfl_xor_sync(0xffffffffu, t, o) : 0.f;
            merge(m2, s2, t2, k);
        }
    }
};

}  // namespace kfac
