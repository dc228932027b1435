// checkpoint.cu -- matrices kept in 8 bits (kfac_checkpoint_store) and restored
// (kfac_checkpoint_load).
//
// A block is 32 consecutive rows of one column: every later use sums over rows (the
// weight gradient, the Kronecker factor), so a block is one K block of a block-scaled
// tensor-core product, which applies the block's power of two itself.  With a the
// block's largest finite magnitude, the exponent is the smallest e >= -127 with
// a <= 448 2^e (448 the largest e4m3 value), and an element is x 2^-e rounded to e4m3:
// the scaling is exact, so an element has the one rounding of e4m3.
//
// Bound by memory.  A CTA takes a tile of 128 rows: each of its four warps 32 rows.  In whole tiles on
// 16-byte boundaries half a warp takes a row's 16-byte groups, 16 rows to a thread, so that a thread has 16
// loads in flight and the maximum over a block is one exchange between two lanes; the tile's
// exponents leave as one piece of 512 bytes.  CTAs next to one another take tiles next to one another in the
// same rows, so that memory is met in long runs.
#include <algorithm>
#include <cstring>

#include "internal.h"
#include "logits.cuh"

namespace kfac {
namespace {

constexpr int TILE = 128;  // rows and columns of a tile of exponents
constexpr int THREADS = 128;
constexpr int MAX_ITEMS = 64;

struct Item {
    char *x;  // source, or where the values go
    long long ld_bytes;
    uint8_t *q;
    long long ldq;
    uint8_t *scales;
    long long rows;
    long long tile_begin;
    int cols, width;  // of x, of the checkpoint (a column of ones more, or not)
    int chunks, wides;  // tiles along the rows and the columns
    int dtype;
    int wide;         // 16-byte accesses to x (8-byte, or 4-byte for 32-bit values, to q)
};
struct Params {
    Item item[MAX_ITEMS];
    int n;
};

__device__ __forceinline__ const Item &item_of(const Params &P, long long tile) {
    int lo = 0, hi = P.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.item[mid].tile_begin <= tile) lo = mid;
        else hi = mid - 1;
    }
    return P.item[lo];
}

// Largest magnitudes, as bits (of finite values the larger bits are the larger value,
// and those of infinities and NaN are larger still).
template <int DT>
struct Mag;
template <>
struct Mag<KFAC_F32> {
    static constexpr uint32_t TOP = 0x7f800000u;
    static __device__ __forceinline__ uint32_t raise(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }
    static __device__ __forceinline__ uint32_t finite(uint32_t w) { return (w & 0x7fffffffu) >= TOP ? 0u : w; }
    static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return max(a, b); }
    static __device__ __forceinline__ uint32_t bits(const uint32_t *m, int i) { return m[i]; }
    static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b); }
};
template <int DT>
struct Mag16 {
    static constexpr uint32_t TOP = DT == KFAC_BF16 ? 0x7f80u : 0x7c00u;
    static __device__ __forceinline__ uint32_t raise(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
    static __device__ __forceinline__ uint32_t finite(uint32_t w) {
        return w & ~__vcmpgeu2(w & 0x7fff7fffu, TOP | TOP << 16);
    }
    static __device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
    static __device__ __forceinline__ uint32_t bits(const uint32_t *m, int i) { return m[i / 2] >> (i & 1) * 16 & 0xffffu; }
    static __device__ __forceinline__ float value(uint32_t b) { return Elem<DT>::value((uint16_t)b); }
};
template <>
struct Mag<KFAC_BF16> : Mag16<KFAC_BF16> {};
template <>
struct Mag<KFAC_F16> : Mag16<KFAC_F16> {};

// The biased exponent (e + 127) of a block whose largest finite magnitude is a.
// 448 = 1.75 2^8: a mantissa above 1.75 takes the next power of two.
__device__ __forceinline__ uint32_t exponent_of(float a) {
    const int k = (int)((__float_as_uint(a) + 0x1fffffu) >> 23);
    return (uint32_t)max(k - 8, 0);
}
// 2^-e from e + 127 (0 .. 247).
__device__ __forceinline__ float inverse_of(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// 2^e (2^-127 is below fp32's normal numbers).
__device__ __forceinline__ float power_of(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x400000u); }
// Past this exponent 256 2^e is infinite in fp32: a value may be rounded up to 240 2^e at most.
constexpr uint32_t LAST_EXPONENT = 247;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// Values that the fast way does not take: an infinity is kept as NaN, and in the last
// exponent a value does not pass 240.
__device__ __forceinline__ float bounded(float y, uint32_t b) {
    if (!(fabsf(y) <= F32_MAX)) return __uint_as_float(0x7fffffffu);
    return b == LAST_EXPONENT ? fminf(fmaxf(y, -240.f), 240.f) : y;
}

// The place of column c's exponents in a tile's (16 bytes to a column modulo 32, 4 to each of 4).
__device__ __forceinline__ int place_of(int c) { return c % 32 * 4 + c % TILE / 32; }

// 16 N columns of a tile, by all its warps, where all its rows and columns are x's and x's rows start
// on 16-byte boundaries: nothing is looked at row by row (otherwise 12.8 instructions an element held it at
// 5.5 TB/s).
template <int DT>
__device__ __forceinline__ void store_whole(const Item &it, long long rt, int cp, uint8_t (*exps)[4]) {
    using M = Mag<DT>;
    constexpr int N = Elem<DT>::N, ROWS = 16;
    using bits = typename Elem<DT>::bits;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long long r0 = rt * TILE + warp * 32 + lane / 16;  // rows r0, r0 + 2, ...
    const int c0 = cp + lane % 16 * N;
    uint4 u[ROWS];
    const char *src = it.x + r0 * it.ld_bytes + (long long)c0 * (int)sizeof(bits);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) u[i] = ld16(src + 2 * i * it.ld_bytes);
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        m[0] = M::raise(m[0], u[i].x); m[1] = M::raise(m[1], u[i].y);
        m[2] = M::raise(m[2], u[i].z); m[3] = M::raise(m[3], u[i].w);
    }
    bool odd = false;
#pragma unroll
    for (int w = 0; w < 4; ++w) m[w] = M::join(m[w], __shfl_xor_sync(ALL_LANES, m[w], 16));
#pragma unroll
    for (int j = 0; j < N; ++j) odd |= M::bits(m, j) >= M::TOP;
    if (__any_sync(ALL_LANES, odd)) {  // infinities or NaN: the largest of the finite ones
        m[0] = m[1] = m[2] = m[3] = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            m[0] = M::raise(m[0], M::finite(u[i].x)); m[1] = M::raise(m[1], M::finite(u[i].y));
            m[2] = M::raise(m[2], M::finite(u[i].z)); m[3] = M::raise(m[3], M::finite(u[i].w));
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) m[w] = M::join(m[w], __shfl_xor_sync(ALL_LANES, m[w], 16));
    }
    uint32_t e[N];
    float inv[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        e[j] = exponent_of(M::value(M::bits(m, j)));
        odd |= e[j] == LAST_EXPONENT;
        inv[j] = inverse_of(e[j]);
    }
    odd = __any_sync(ALL_LANES, odd);
    uint8_t *dst = it.q + r0 * it.ldq + c0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        float v[N];
        Elem<DT>::unpack(u[i], v);
        uint32_t b[N / 4];
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= inv[j];
        if (odd) {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = bounded(v[j], e[j]);
        }
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
            b[j] = e4m3x2(v[4 * j], v[4 * j + 1]) | e4m3x2(v[4 * j + 2], v[4 * j + 3]) << 16;
        // (q's rows start on 16-byte boundaries, and c0 is a multiple of N)
        if constexpr (N == 8) *(uint2 *)(dst + 2 * i * it.ldq) = make_uint2(b[0], b[1]);
        else *(uint32_t *)(dst + 2 * i * it.ldq) = b[0];
    }
    if (lane < 16) {
#pragma unroll
        for (int j = 0; j < N; ++j) exps[place_of(c0 + j)][warp] = (uint8_t)e[j];
    }
}

// A value by itself.
template <int DT>
__device__ __forceinline__ float value_of(uint32_t b) {
    if constexpr (DT == KFAC_F32) return __uint_as_float(b);
    else return Elem<DT>::value((uint16_t)b);
}

// A whole tile at any alignment, whatever part of it is x's: a column to a lane, 32 rows to a warp, 32 columns
// at a time (2 groups of them in flight), value by value.  A block is a lane's own then, and an instruction
// meets 32 values side by side.
template <int DT>
__device__ __forceinline__ void store_columns(const Item &it, long long rt, int ct, uint8_t (*exps)[4]) {
    using bits = typename Elem<DT>::bits;
    constexpr int GROUPS = 2;
    constexpr uint32_t SIGN = DT == KFAC_F32 ? 0x80000000u : 0x8000u, TOP = Mag<DT>::TOP;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long long r0 = rt * TILE + warp * 32;
    const int rows = (int)max(0LL, min(32LL, it.rows - r0));
#pragma unroll 1
    for (int g = 0; g < TILE / 32; g += GROUPS) {
        uint32_t w[GROUPS][32];
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
            const int c = ct * TILE + (g + k) * 32 + lane;
            const char *p = it.x + r0 * it.ld_bytes + (long long)c * (int)sizeof(bits);
            const int here = c < it.cols ? rows : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                w[k][i] = 0;
                if (i < here) w[k][i] = *(const bits *)p;
                p += it.ld_bytes;
            }
        }
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
            const int c = ct * TILE + (g + k) * 32 + lane;
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) m = max(m, w[k][i] & ~SIGN);
            bool odd = m >= TOP;
            if (__any_sync(ALL_LANES, odd)) {  // infinities or NaN: the largest of the finite ones
                m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) m = max(m, (w[k][i] & ~SIGN) >= TOP ? 0u : w[k][i] & ~SIGN);
            }
            const uint32_t e = exponent_of(value_of<DT>(m));
            const float inv = inverse_of(e);
            odd = __any_sync(ALL_LANES, odd || e == LAST_EXPONENT);
            uint8_t *d = it.q + r0 * it.ldq + c;
            const int here = c < it.width ? rows : 0;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float v0 = value_of<DT>(w[k][i]) * inv, v1 = value_of<DT>(w[k][i + 1]) * inv;
                if (odd) {
                    v0 = bounded(v0, e);
                    v1 = bounded(v1, e);
                }
                const uint32_t b = c == it.cols ? 0x7878u : e4m3x2(v0, v1);  // a one: 256 2^-8
                if (i < here) *d = (uint8_t)b;
                d += it.ldq;
                if (i + 1 < here) *d = (uint8_t)(b >> 8);
                d += it.ldq;
            }
            exps[place_of(c)][warp] = (uint8_t)(here == 0 ? 0u : c < it.cols ? e : 119u);  // 1 = 256 2^-8
        }
    }
}

template <int DT>
__device__ __forceinline__ void store_tile(const Item &it, long long tile, uint8_t (*exps)[4]) {
    constexpr int COLS = 16 * Elem<DT>::N;
    const int ct = (int)(tile % it.wides);
    const long long rt = tile / it.wides;
    if (it.wide && (rt + 1) * TILE <= it.rows && (ct + 1) * TILE <= it.cols) {
#pragma unroll 1
        for (int cp = ct * TILE; cp < (ct + 1) * TILE; cp += COLS) store_whole<DT>(it, rt, cp, exps);
    } else {
        store_columns<DT>(it, rt, ct, exps);
    }
    __syncthreads();
    ((uint32_t *)(it.scales + (ct * (long long)it.chunks + rt) * 512))[threadIdx.x] = ((const uint32_t *)exps)[threadIdx.x];
}

// 32768 x 8192 16-bit values (814 MB) take 115 us, 7.1 TB/s (a copy: 6.8); 20000 x 5001 (rows on every
// alignment) 77 us, 3.9 TB/s, 16384 x 4097 fp32 63, 5.3 TB/s, 1000 x 1001 4.4.  With five CTAs to an SM or one group
// in flight 106 and 138, 97 and 100, 7 and 9; by 16 bytes with the rest of a group from the next lane
// 74, 76 and 11.
__global__ void __launch_bounds__(THREADS, 4) store_kernel(const __grid_constant__ Params P) {
    __shared__ __align__(16) uint8_t exps[TILE][4];
    pdl_wait();
    pdl_trigger();
    const Item &it = item_of(P, blockIdx.x);
    const long long tile = blockIdx.x - it.tile_begin;
    if (it.dtype == KFAC_BF16) store_tile<KFAC_BF16>(it, tile, exps);
    else if (it.dtype == KFAC_F16) store_tile<KFAC_F16>(it, tile, exps);
    else store_tile<KFAC_F32>(it, tile, exps);
}

// 16 bytes from byte k (0 .. 15) of 32.
__device__ __forceinline__ uint4 from_byte(uint4 lo, uint4 hi, int k) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = k & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = k & 4 ? w[i + 1] : w[i];
    const int s = (k & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}

// Elements j0 .. j1 - 1 of a group.  (In pieces of 2, 4 and 8 bytes, fewer but other ones for either end of a
// row's part: 20000 x 5001 in 83 us in place of 69.)
template <int DT>
__device__ __forceinline__ void store_some(char *d, uint4 u, int j0, int j1) {
    using bits = typename Elem<DT>::bits;
    constexpr int N = Elem<DT>::N;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j >= j0 && j < j1) ((bits *)d)[j] = (bits)(N == 4 ? w[j] : w[j / 2] >> (j & 1) * 16);
}
// The first `n` elements (0 .. N) of a group to a 16-byte boundary.
template <int DT>
__device__ __forceinline__ void store_first(char *d, uint4 u, int n) {
    constexpr int PER = Elem<DT>::N / 4;  // to a word
    if (n >= 4 * PER) {
        *(uint4 *)d = u;
        return;
    }
    if (n & 2 * PER) {
        *(uint2 *)d = make_uint2(u.x, u.y);
        u.x = u.z;
        u.y = u.w;
        d += 8;
    }
    if (n & PER) {
        *(uint32_t *)d = u.x;
        u.x = u.y;
        d += 4;
    }
    if (PER == 2 && n & 1) *(uint16_t *)d = (uint16_t)u.x;
}
// The last `n` elements (1 .. N - 1) of one.
template <int DT>
__device__ __forceinline__ void store_last(char *d, uint4 u, int n) {
    constexpr int N = Elem<DT>::N, PER = N / 4;
    const int j = N - n;
    if (PER == 2 && n & 1) ((uint16_t *)d)[j] = (uint16_t)((j & 4 ? j & 2 ? u.w : u.z : j & 2 ? u.y : u.x) >> 16);
    if (n & PER) ((uint32_t *)d)[n & 2 * PER ? 1 : 3] = n & 2 * PER ? u.y : u.w;
    if (n & 2 * PER) ((uint2 *)d)[1] = make_uint2(u.z, u.w);
}
// Elements j0 .. j1 - 1 of one.
template <int DT>
__device__ __noinline__ void store_between(char *d, uint4 u, int j0, int j1) {
    using bits = typename Elem<DT>::bits;
    constexpr int N = Elem<DT>::N;
#pragma unroll 1
    for (int j = 0; j < j1; ++j) {
        if (j >= j0) ((bits *)d)[j] = (bits)u.x;
        constexpr int S = 128 / N % 32;
        u = S ? make_uint4(__funnelshift_r(u.x, u.y, S), __funnelshift_r(u.y, u.z, S), __funnelshift_r(u.z, u.w, S), u.w >> S)
              : make_uint4(u.y, u.z, u.w, 0);
    }
}

// The rows that half a warp has of a tile, at most 16.
__device__ __forceinline__ int rows_of(const Item &it, long long rt, int warp) {
    return (int)max(0LL, min(16LL, (it.rows - (rt * TILE + warp * 32) + 1) / 2));
}

// Values of 16 N columns of a tile, x_ij = q_ij 2^e, rounded to x's type.  FULL: all rows and columns are
// x's, and nothing is looked at row by row; other parts go four rows at a time in short code, most of whose
// time is its fetching (1000 x 1000 4 us, with all rows unrolled 7).  A column to a lane, as in store_columns, takes
// 2.5 times as long: the pieces of sectors that are written then.
template <int DT, bool FULL>
__device__ __forceinline__ void load_part(const Item &it, long long rt, int cp, const uint8_t (*exps)[4]) {
    constexpr int N = Elem<DT>::N, ROWS = FULL ? 16 : 4;
    using bits = typename Elem<DT>::bits;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    long long r0 = rt * TILE + warp * 32 + lane / 16;
    const int c0 = cp + lane % 16 * N;
    const int n = FULL ? N : max(0, min(N, it.cols - c0));  // values here
    const int rows = FULL ? 16 : cp >= it.cols ? 0 : rows_of(it, rt, warp);
    float p[N];
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = power_of(exps[place_of(c0 + j)][warp]);
    // At other alignments a lane stores the 16 bytes that its group begins in, with the last elements of the
    // group of the lane before it; the last lane of a row's part stores what is left of its own, too.
    const bool begin = lane % 16 == 0, end = FULL ? lane % 16 == 15 : lane % 16 == 15 || c0 + N >= it.cols;
#pragma unroll 1
    for (int k = 0; k < rows; k += ROWS, r0 += 2 * ROWS) {
        const uint8_t *src = it.q + r0 * it.ldq + c0;
        char *dst = it.x + r0 * it.ld_bytes + (long long)c0 * (int)sizeof(bits);
        uint32_t b[ROWS][N / 4];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            b[i][0] = b[i][N / 4 - 1] = 0;
            if (!FULL && (r0 + 2 * i >= it.rows || n == 0)) continue;  // (a group with a value in it is read whole)
            if constexpr (N == 8) {
                const uint2 u = *(const uint2 *)(src + 2 * i * it.ldq);
                b[i][0] = u.x;
                b[i][1] = u.y;
            } else {
                b[i][0] = *(const uint32_t *)(src + 2 * i * it.ldq);
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            float v[N];
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const float2 f = from_e4m3x2(b[i][j / 4] >> j % 4 * 8 & 0xffffu);
                v[j] = f.x * p[j];
                v[j + 1] = f.y * p[j + 1];
            }
            char *d = dst + 2 * i * it.ld_bytes;
            const uint4 u = Elem<DT>::pack(v);
            const bool in = FULL || (r0 + 2 * i < it.rows && n > 0);
            if (it.wide) {
                if (in) store_first<DT>(d, u, n);
                continue;
            }
            constexpr int SIZE = (int)sizeof(bits);
            const int off = (int)((uintptr_t)d & 15), skip = off / SIZE;  // elements of the 16 bytes that are before the group
            uint4 before = make_uint4(__shfl_up_sync(ALL_LANES, u.x, 1, 16), __shfl_up_sync(ALL_LANES, u.y, 1, 16),
                                      __shfl_up_sync(ALL_LANES, u.z, 1, 16), __shfl_up_sync(ALL_LANES, u.w, 1, 16));
            if (!in) continue;
            if (FULL) {
                if (off == 0) *(uint4 *)d = u;
                else if (!begin) *(uint4 *)(d - off) = from_byte(before, u, 16 - off);
                if (off && (begin || end)) store_some<DT>(d, u, begin ? 0 : N - skip, begin ? N - skip : N);
                continue;
            }
            if (off == 0) before = u;
            const uint4 g = from_byte(before, u, 16 - off & 15);
            const int to = min(N, skip + n);
            if (!begin || skip == 0) store_first<DT>(d - off, g, to);
            else if (to == N) store_last<DT>(d - off, g, N - skip);
            else store_between<DT>(d - off, g, skip, to);
            if (end && skip + n > N) store_first<DT>(d - off + 16, from_byte(u, make_uint4(0, 0, 0, 0), 16 - off & 15), skip + n - N);
        }
    }
}

template <int DT>
__device__ __forceinline__ void load_tile(const Item &it, long long tile, const uint8_t (*exps)[4]) {
    constexpr int COLS = 16 * Elem<DT>::N;
    const int ct = (int)(tile % it.wides);
    const long long rt = tile / it.wides;
    const bool rows = (rt + 1) * TILE <= it.rows;
#pragma unroll 1
    for (int cp = ct * TILE; cp < (ct + 1) * TILE; cp += COLS) {
        if (rows && cp + COLS <= it.cols) load_part<DT, true>(it, rt, cp, exps);
        else load_part<DT, false>(it, rt, cp, exps);
    }
}

// 32768 x 8192 16-bit values take 117 us, 6.9 TB/s (six CTAs to an SM 119); 20000 x 5001 70 us; 1000 x 1000,
// most of whose tiles are not whole, 4.
__global__ void __launch_bounds__(THREADS, 5) load_kernel(const __grid_constant__ Params P) {
    __shared__ __align__(16) uint8_t exps[TILE][4];
    pdl_wait();
    pdl_trigger();
    const Item &it = item_of(P, blockIdx.x);
    const long long tile = blockIdx.x - it.tile_begin;
    const long long at = tile % it.wides * it.chunks + tile / it.wides;
    ((uint32_t *)exps)[threadIdx.x] = ((const uint32_t *)(it.scales + at * 512))[threadIdx.x];
    __syncthreads();
    if (it.dtype == KFAC_BF16) load_tile<KFAC_BF16>(it, tile, exps);
    else if (it.dtype == KFAC_F16) load_tile<KFAC_F16>(it, tile, exps);
    else load_tile<KFAC_F32>(it, tile, exps);
}

size_t elem_size(int dtype) { return dtype == KFAC_F32 ? 4 : 2; }

kfac_status check(const kfac_checkpoint_desc *descs, int count) {
    if (count < 0 || (count > 0 && !descs)) return KFAC_ERR_INVALID;
    for (int i = 0; i < count; ++i) {
        const kfac_checkpoint_desc &d = descs[i];
        if (d.dtype != KFAC_BF16 && d.dtype != KFAC_F16 && d.dtype != KFAC_F32) return KFAC_ERR_INVALID;
        if (d.rows < 0 || d.cols < 1 || d.ld < d.cols || (uintptr_t)d.x % elem_size(d.dtype)) return KFAC_ERR_INVALID;
        const kfac_status s =
            check_checkpoint(d.q, d.ldq, d.scales, d.rows, (long long)d.cols + (d.append_one ? 1 : 0));
        if (s != KFAC_OK) return s;
        if (d.rows > 0 && !d.x) return KFAC_ERR_INVALID;
    }
    return KFAC_OK;
}

kfac_status run(const kfac_checkpoint_desc *descs, int count, bool store, void *stream) {
    kfac_status s = check(descs, count);
    if (s != KFAC_OK) return s;
    DeviceMemory memory;
    for (int i = 0; i < count; ++i)
        if (descs[i].rows > 0 && !(memory.holds(descs[i].x, 0) && memory.holds(descs[i].q, 1) && memory.holds(descs[i].scales, 2)))
            return KFAC_ERR_INVALID;
    cudaStream_t st = (cudaStream_t)stream;
    for (int at = 0; at < count;) {
        Params P;
        P.n = 0;
        long long tiles = 0;
        while (at < count && P.n < MAX_ITEMS) {
            const kfac_checkpoint_desc &d = descs[at];
            const long long chunks = ceil_div(d.rows, TILE), width = d.cols + (d.append_one ? 1 : 0);
            // (what is only restored may leave the ones' tile out; it is kept, so that a tile's number is its place)
            const long long here = chunks * ceil_div(width, TILE);
            if (here == 0) {
                ++at;
                continue;
            }
            if (tiles + here > 0x7fffffffLL) break;  // (one item alone stays below: check_checkpoint)
            Item &it = P.item[P.n++];
            it.x = (char *)d.x;
            it.ld_bytes = d.ld * (long long)elem_size(d.dtype);
            it.q = d.q;
            it.ldq = d.ldq;
            it.scales = d.scales;
            it.rows = d.rows;
            it.tile_begin = tiles;
            it.cols = d.cols;
            it.width = (int)width;
            it.chunks = (int)chunks;
            it.wides = (int)ceil_div(width, TILE);
            it.dtype = d.dtype;
            it.wide = (uintptr_t)d.x % 16 == 0 && (it.ld_bytes % 16 == 0 || d.rows == 1);
            tiles += here;
            ++at;
        }
        if (P.n == 0) break;
        if (store) KFAC_LAUNCH(KK_CHECKPOINT, st, store_kernel, (unsigned)tiles, THREADS, 0, P);
        else KFAC_LAUNCH(KK_CHECKPOINT, st, load_kernel, (unsigned)tiles, THREADS, 0, P);
    }
    return KFAC_OK;
}

}  // namespace

// What every call that takes a checkpoint checks of it: elements on 16-byte rows, whole
// tiles of exponents.
kfac_status check_checkpoint(const void *q, long long ldq, const void *scales, long long rows, long long width) {
    if (rows < 0 || width < 1 || (rows > 0 && (!q || !scales || ldq < width))) return KFAC_ERR_INVALID;
    if (rows > 0x7fffffffLL || width > (1 << 20) || ceil_div(rows, TILE) * ceil_div(width, TILE) > 0x7fffffffLL)
        return KFAC_ERR_UNSUPPORTED;
    if (rows > 0 && (ldq % 16 || (uintptr_t)q % 16 || (uintptr_t)scales % 16)) return KFAC_ERR_UNSUPPORTED;
    return KFAC_OK;
}

}  // namespace kfac

extern "C" size_t kfac_checkpoint_scale_bytes(int64_t rows, int32_t width) {
    if (rows < 0 || width < 1) return 0;
    return (size_t)kfac::ceil_div(rows, 128) * (size_t)kfac::ceil_div(width, 128) * 512;
}

extern "C" kfac_status kfac_checkpoint_store(const kfac_checkpoint_desc *descs, int count, void *stream) {
    return kfac::run(descs, count, true, stream);
}

extern "C" kfac_status kfac_checkpoint_load(const kfac_checkpoint_desc *descs, int count, void *stream) {
    return kfac::run(descs, count, false, stream);
}
