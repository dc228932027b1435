// mx_gemm.cu -- products of two checkpoints over their rows, C = beta C + alpha A^T B,
// on the block-scaled tensor cores (tcgen05, kind::mxf8f6f4): e4m3 elements, a power of
// two for each 32 rows of a column.
//
// Both operands are read as they are stored, rows of tokens with the features side by
// side, so both are MN-major; 32 tokens are one K step of the product and one block of
// exponents.  The tensor core multiplies exactly and adds in fp32; sums over more than
// CHUNK tokens are added up in registers with fp32's own rounding, because a long sum in
// one tensor-core accumulator loses bits.
//
// A persistent kernel, a pair of CTAs (two SMs) to a tile of 256 x 256: each brings half of
// both operands, and the pair's products (cta_group::2) read both halves, so that a byte
// brought to an SM serves 128 products (a tile of 128 x 128 on one SM: 64, and the
// operands' way to the SMs held it at 1.46 PFLOP/s).  In each CTA one warp brings operand tiles
// by TMA and eight take the accumulator out of tensor memory into registers at once, so that
// the next tile's products start before this one's stores; one thread of the first CTA issues
// the products of both.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <memory>
#include <type_traits>
#include <vector>

#include "internal.h"
#include "mx_plan.h"

namespace kfac {
namespace {

constexpr int HALF = 128, TILE = 2 * HALF, BK = 128;  // a CTA's rows, the pair's tile, tokens a stage
using namespace mx;  // how the tiles are dealt out to the pairs
constexpr int STAGES = 5;
constexpr int TILE_BYTES = 128 * 128, SF_BYTES = 512;
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int SF_STAGE = 3 * SF_BYTES;  // a stage's exponents: of the CTA's rows, and of all columns
// Four warps (two of them idle) and eight with the accumulator in registers: the register
// file is split 56 : 224 : 224 a thread among the three groups of four (504 = 3 * 168 at launch).
constexpr int EPI_WARPS = 8, FIRST_EPI = 4, NUM_THREADS = 32 * (FIRST_EPI + EPI_WARPS);
constexpr int FEW_REGS = 56, MANY_REGS = 224;
constexpr int COLS = TILE / 2;  // accumulator columns of an epilogue warp
constexpr int LD = 36;        // pitch of its staging chunk
// Tensor memory: the accumulator at column 0 and, of every other chunk, at column 192, so that
// a chunk's products may start when the 64 columns that both have are taken out of the one
// before; and the exponents, a slot for each stage.
constexpr int ACC_SHIFT = 192, SF_COL = 448, SF_SLOT = 12;
static_assert(SF_COL + STAGES * SF_SLOT <= 512 && ACC_SHIFT + TILE <= SF_COL && TILE - ACC_SHIFT == 64, "tensor memory");
constexpr int TMEM_COLS = 512;
// Stages (1280 tokens) in one accumulator.  Sums of 2048 to 20000 tokens are off by at most 9e-7 of
// themselves (8 stages 7e-7, 16 stages 1.6e-6, 64 stages 3e-6 to 7e-6), and taking a chunk out costs 0.9 us
// (16384 x 4096 x 8192: 8 stages 426 us, 10 stages 395, 16 stages 354).  Three accumulators of half a
// tile that are taken out in turn wait less, but their products of 128 columns read A twice from shared
// memory (391 us; 2048 x 4096 x 4096 48 in place of 41).
constexpr int CHUNK = 10;
constexpr size_t SMEM_BYTES =
    1024 + STAGES * (STAGE_BYTES + SF_STAGE) + EPI_WARPS * 32 * LD * sizeof(float) + 256;

struct Maps {
    CUtensorMap a, b, sa, sb;  // elements and exponents
};
struct Prob : Maps, Tiles {
    void *C;
    long long ldc;
    int M, N;
    float alpha, beta;
    uint8_t packed, c_dtype, vec;
};
// CAP: room for problems.  A kernel's parameters are copied at its launch (30 KB of them for
// about 3 us), so that few problems have a kernel of their own.
template <int CAP>
struct Params : Deal {
    Prob prob[CAP];
    float *partial;  // [2 pairs][TILE][TILE] pieces of tiles: 2 p begins inside a tile, 2 p + 1 ends inside one
    int *counters;   // [pairs][2][EPI_WARPS] pieces that are there of the tile that the pair's share ends in, by CTA and warp
    int *err;
    bool alone;      // one pair, which sets *err to 0 (no one else writes it)
};
constexpr int FEW_PROBS = 4;
static_assert(sizeof(Params<MAX_PROBS>) <= 32000, "kernel parameters");

// Shared-memory descriptor of a slice of 32 tokens: groups of 8 rows of 128 features,
// 128-byte swizzle, 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t tile, int slice) {
    return smem_desc_sw128(tile + slice * 4096, TILE_BYTES, 1024);
}
// Of 512 bytes of exponents: 32 rows of 16 bytes, groups of 8 rows 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t exponents(uint32_t at) {
    return (uint64_t)((at & 0x3FFFF) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// Copies them to four columns of tensor memory, the same for each quarter of the lanes; in
// both CTAs, each its own.
__device__ __forceinline__ void copy_exponents(uint32_t tmem, uint32_t smem) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(exponents(smem)) : "memory");
}
// Instruction descriptor: e4m3 operands, both MN-major, fp32 accumulator, exponents as
// powers of two; `slice` is the byte of a column of exponents.
__device__ __forceinline__ uint32_t idesc(int M, int N, int slice) {
    return (uint32_t)slice << 4 | 1u << 15 | 1u << 16 | (uint32_t)(N >> 3) << 17 | 1u << 23 | (uint32_t)(M >> 4) << 24 |
           (uint32_t)slice << 29;
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                    uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` of both CTAs when every product issued so far is done.
__device__ __forceinline__ void commit_both(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// The address of the first CTA's copy of a shared variable.
__device__ __forceinline__ uint32_t of_first(const void *p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(0));
    return a;
}
// A tile into this CTA's shared memory, its bytes counted on the first CTA's barrier.
__device__ __forceinline__ void load_pair(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *slot) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t at) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(TMEM_COLS) : "memory");
}

__device__ __forceinline__ float from_16(uint32_t b, bool f16) {
    return f16 ? __half2float(__ushort_as_half((uint16_t)b)) : bf16_bits_to_f32((uint16_t)b);
}


// The part inside the result (on and above the diagonal of a symmetric one) of 32 rows x 32
// columns at (i0, j0): a column to a lane, a row to an instruction, at any pitch or packing.
// Short loops: what it takes is mostly the fetching of its code (a chunk 6.5 us with
// the types told apart at every row and 16 rows unrolled).
template <int DT>
__device__ __forceinline__ bool store_edge(const Prob &q, int i0, int j0, float *stage, int lane) {
    using T = std::conditional_t<DT == KFAC_F32, float, uint16_t>;
    const int j = j0 + lane, rows = min(32, q.M - i0);
    const int n = j >= q.N ? 0 : q.sym ? min(rows, j - i0 + 1) : rows;  // rows of this lane's column
    // a packed triangle's row i starts (j counted from 0) at i N - i (i + 1) / 2
    const int shorter = q.packed ? 1 : 0;
    const long long first = (shorter ? (long long)i0 * q.N - (long long)i0 * (i0 + 1) / 2 : (long long)i0 * q.ldc) + j;
    const long long pitch = shorter ? q.N - 1 - i0 : q.ldc;  // to the next row, one less each time in a triangle
    T *C = (T *)q.C;
    float scale = q.alpha;
    if (const float beta = q.beta; beta != 0.f) {
        long long at = first, to = pitch;
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += 16) {
            T old[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                old[r] = T(0);
                if (r0 + r < n) old[r] = C[at];
                at += to;
                to -= shorter;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float &v = stage[(r0 + r) * LD + lane];
                if constexpr (DT == KFAC_F32) v = fmaf(beta, old[r], scale * v);
                else v = fmaf(beta, from_16(old[r], DT == KFAC_F16), scale * v);
            }
        }
        scale = 1.f;
    }
    bool bad = false;
    long long at = first, to = pitch;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
        const float v = scale * stage[r * LD + lane];
        if (r < n) {
            bad |= !(fabsf(v) <= 3.402823466e38f);
            if constexpr (DT == KFAC_F32) C[at] = v;
            else C[at] = f32_to_16_bits(v, DT == KFAC_F16);
        }
        at += to;
        to -= shorter;
    }
    return bad;
}

// Stores the 32 rows x 32 columns at (i0, j0) that a warp has in its stage (pitch LD).
// Returns whether a value was NaN or infinite.  Chunks inside the result whose rows start on
// 16-byte boundaries (8-byte ones of 16-bit values) go four values to a lane, four rows to an
// instruction; others go through store_edge.
__device__ __forceinline__ bool store_chunk(const Prob &q, int i0, int j0, float *stage, int lane) {
    bool bad = false;
    if (j0 >= q.N || i0 >= q.M || (q.sym && j0 + 31 < i0)) return false;
    const float alpha = q.alpha, beta = q.beta;
    if (q.vec && i0 + 32 <= q.M && j0 + 32 <= q.N && (!q.sym || j0 >= i0 + 32)) {
        const int r = lane >> 3, c = 4 * (lane & 7);
        const long long ldc = q.ldc, at = (long long)(i0 + r) * ldc + j0 + c, step = 4 * ldc;
        if (q.c_dtype == KFAC_F32) {
            float *dst = (float *)q.C + at;
            float4 old[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                old[k] = beta != 0.f ? *(const float4 *)(dst + k * step) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 v = *(const float4 *)(stage + (4 * k + r) * LD + c);
                const float4 o = make_float4(fmaf(beta, old[k].x, alpha * v.x), fmaf(beta, old[k].y, alpha * v.y),
                                             fmaf(beta, old[k].z, alpha * v.z), fmaf(beta, old[k].w, alpha * v.w));
                bad |= !finite4(o);
                *(float4 *)(dst + k * step) = o;
            }
        } else {
            uint16_t *dst = (uint16_t *)q.C + at;
            const bool h = q.c_dtype == KFAC_F16;
            uint2 old[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) old[k] = beta != 0.f ? *(const uint2 *)(dst + k * step) : make_uint2(0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 v = *(const float4 *)(stage + (4 * k + r) * LD + c);
                const float4 o =
                    make_float4(fmaf(beta, from_16(old[k].x, h), alpha * v.x), fmaf(beta, from_16(old[k].x >> 16, h), alpha * v.y),
                                fmaf(beta, from_16(old[k].y, h), alpha * v.z), fmaf(beta, from_16(old[k].y >> 16, h), alpha * v.w));
                bad |= !finite4(o);
                *(uint2 *)(dst + k * step) =
                    make_uint2(f32_to_16_bits(o.x, h) | (uint32_t)f32_to_16_bits(o.y, h) << 16,
                               f32_to_16_bits(o.z, h) | (uint32_t)f32_to_16_bits(o.w, h) << 16);
            }
        }
        return bad;
    }
    if (q.c_dtype == KFAC_F32) return store_edge<KFAC_F32>(q, i0, j0, stage, lane);
    if (q.c_dtype == KFAC_F16) return store_edge<KFAC_F16>(q, i0, j0, stage, lane);
    return store_edge<KFAC_BF16>(q, i0, j0, stage, lane);
}

__device__ __forceinline__ bool all_of(bool ok) { return __all_sync(0xffffffffu, ok); }
// True on one lane of a warp that is here as a whole.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
// The warp has read what the next chunk's accumulator overlaps.
__device__ __forceinline__ void released_by(uint32_t bar, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_at(bar);
}
template <int AT>
__device__ __forceinline__ void add_columns(float (&v)[COLS], const float (&t)[32], const Item &k) {
    if (k.kt0 >= k.kt1) return;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[AT + i] += t[i];
}

template <int CAP>
__global__ void __launch_bounds__(NUM_THREADS, 1) mx_kernel(const __grid_constant__ Params<CAP> P) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sf = smem + STAGES * STAGE_BYTES;
    float *stages = (float *)(sf + STAGES * SF_STAGE);
    uint64_t *full = (uint64_t *)(stages + EPI_WARPS * 32 * LD);
    uint64_t *empty = full + STAGES;
    uint64_t *accf = empty + STAGES, *acce = accf + 1, *drain = acce + 1;
    uint32_t *tmem_slot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, rank = blockIdx.x & 1;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accf, 1);
        mbar_init(acce, 2 * EPI_WARPS);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot);
    if (warp == 2 && lane < 4 && P.prob[0].k_tiles > 0) tma_prefetch_desc(&P.prob[0].a + lane);  // (without rows there are none)
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp < FIRST_EPI) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FEW_REGS));
        // The whole of a warp runs its loop and one of its threads issues: what copies and products
        // take (addresses, descriptors) is then the same for all lanes to the compiler, too.  Issued from
        // a thread's own branch a stage's products took 0.45 us, more than the tensor cores do.
        if (warp == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            bool ok = true;
            Walk walk(P, pair, pairs);
            for (Item k; ok && walk.next(P, k);) {
                const Prob &q = P.prob[k.p];
                const bool same = q.sym && k.tm == k.tn;
                const uint32_t bytes = 2 * ((same ? 1 : 2) * TILE_BYTES + SF_STAGE);
                const int i0 = k.tm * TILE + rank * HALF, j0 = k.tn * TILE + rank * HALF, k_tiles = q.k_tiles;
                const int ta = (2 * k.tm + rank) * k_tiles, tb = 2 * k.tn * k_tiles;
                for (int kt = k.kt0; kt < k.kt1; ++kt) {
                    ok = all_of(mbar_wait(&empty[stage], phase ^ 1) && !*abort_flag);
                    if (!ok) {
                        if (lane == 0) atomicOr(P.err, ERR_TIMEOUT_EMPTY);
                        *abort_flag = 1;
                        break;
                    }
                    const uint32_t bar = of_first(&full[stage]);
                    uint8_t *s = smem + stage * STAGE_BYTES, *f = sf + stage * SF_STAGE;
                    if (elect_one()) {
                        // (both CTAs' bytes; the other's may be counted before they are expected)
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);
                        load_pair(s, &q.a, i0, kt * BK, bar);
                        if (!same) load_pair(s + TILE_BYTES, &q.b, j0, kt * BK, bar);
                        load_pair(f, &q.sa, 0, ta + kt, bar);
                        load_pair(f + SF_BYTES, &q.sb, 0, tb + kt, bar);
                        load_pair(f + 2 * SF_BYTES, &q.sb, 0, tb + k_tiles + kt, bar);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    ++issued;
                }
            }
            // cut short: the copies that are on their way land before the CTAs leave (both wait for each other)
            if (!ok && rank == 0) {
                for (int n = 0; n < min(issued, STAGES); ++n) {
                    if (stage == 0) { stage = STAGES - 1; phase ^= 1; } else { --stage; }
                    if (!mbar_wait(&full[stage], phase) && lane == 0) atomicOr(P.err, ERR_TIMEOUT_DRAIN);
                }
            }
            // (those of the second CTA are counted on the first one's barriers, which may not expect them any more:
            // they are given a millisecond, a thousand times what a copy takes)
            if (!ok && rank == 1)
                for (const uint64_t t0 = global_timer_ns(); global_timer_ns() - t0 < 1000000;) __nanosleep(1000);
        }
        if (warp == 1 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0, use = 0;
            bool ok = true;
            const uint32_t s0 = smem_u32(smem), f0 = smem_u32(sf);
            if (P.alone && lane == 0) {  // before the first product, and so before anyone reports
                *P.err = 0;
                __threadfence();
            }
            __syncwarp();
            Walk walk(P, pair, pairs);
            for (Item k; ok && walk.next(P, k);) {
                const Prob &q = P.prob[k.p];
                const bool same = q.sym && k.tm == k.tn;
                for (int c0 = k.kt0; ok; c0 += CHUNK) {
                    const int c1 = min(k.kt1, c0 + CHUNK);
                    ok = all_of(mbar_wait(acce, (use & 1) ^ 1));
                    if (!ok) {
                        if (lane == 0) atomicOr(P.err, ERR_TIMEOUT_ACC);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + (use & 1) * ACC_SHIFT;
                    ++use;
                    for (int kt = c0; kt < c1; ++kt) {
                        ok = all_of(mbar_wait(&full[stage], phase));
                        if (!ok) {
                            if (lane == 0) atomicOr(P.err, ERR_TIMEOUT_FULL);
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a = s0 + stage * STAGE_BYTES, b = same ? a : a + TILE_BYTES, f = f0 + stage * SF_STAGE;
                        const uint32_t ta = tmem + SF_COL + stage * SF_SLOT, tb = ta + 4;
                        if (elect_one()) {
                            // (a slot of exponents is written again when its stage's products are done)
                            copy_exponents(ta, f);
                            copy_exponents(tb, f + SF_BYTES);
                            copy_exponents(tb + 4, f + 2 * SF_BYTES);
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                mma(d, operand(a, s), operand(b, s), idesc(TILE, TILE, s), ta, tb, kt > c0 || s > 0);
                            commit_both(&empty[stage]);
                        }
                        __syncwarp();
                        if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    if (elect_one()) commit_both(accf);
                    __syncwarp();
                    if (c1 >= k.kt1) break;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                if (elect_one()) commit_both(drain);
                __syncwarp();
                if (!mbar_wait(drain, 0) && lane == 0) atomicOr(P.err, ERR_TIMEOUT_DRAIN);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(MANY_REGS));
        const int e = warp - FIRST_EPI, quarter = warp & 3, half = e >> 2;
        // this warp's columns: 32 of each 64 of the tile, v[32 m ..] those of 64 m + 32 half
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + half * 32;
        float *stage = stages + e * 32 * LD;
        const uint32_t released = of_first(acce);
        uint32_t use = 0;
        bool bad = false;
        Walk walk(P, pair, pairs);
        for (Item k; all_of(!*abort_flag) && walk.next(P, k);) {
            const Prob &q = P.prob[k.p];
            const int i0 = k.tm * TILE + rank * HALF + quarter * 32, j0 = k.tn * TILE + half * 32;
            if (q.beta != 0.f && !q.packed && i0 + lane < q.M) {  // the old values on their way to L2 while the products run
                const int size = q.c_dtype == KFAC_F32 ? 4 : 2;
                const char *row = (const char *)q.C + ((long long)(i0 + lane) * q.ldc + j0) * size;
#pragma unroll
                for (int c = 0; c < COLS; c += 32)
                    if (j0 + 2 * c < q.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 2 * c * size));
            }
            float v[COLS];
            bool ok = true;
            for (int c0 = k.kt0;; c0 += CHUNK) {
                if (!all_of(mbar_wait(accf, use & 1))) {  // (the loads from tensor memory want the whole warp)
                    ok = false;
                    break;
                }
                tc_fence_after();
                // (without a token nothing was multiplied: the accumulator holds another tile's values)
                if (c0 == k.kt0) {
#pragma unroll
                    for (int i = 0; i < COLS; ++i) v[i] = 0.f;
                }
                // first what the next chunk's accumulator overlaps: the last 64 columns of one at column 0, the
                // first of one at column 192
                float t[32], u[32];
                if (use & 1) {
                    tmem_ld_32x32b_x32(lanes + ACC_SHIFT, t);
                    released_by(released, lane);
                    add_columns<0>(v, t, k);
                    tmem_ld_pair_32x32b_x32(lanes + ACC_SHIFT + 64, t, lanes + ACC_SHIFT + 128, u);
                    add_columns<32>(v, t, k);
                    add_columns<64>(v, u, k);
                    tmem_ld_32x32b_x32(lanes + ACC_SHIFT + 192, t);
                    add_columns<96>(v, t, k);
                } else {
                    tmem_ld_32x32b_x32(lanes + 192, t);
                    released_by(released, lane);
                    add_columns<96>(v, t, k);
                    tmem_ld_pair_32x32b_x32(lanes + 64, t, lanes + 128, u);
                    add_columns<32>(v, t, k);
                    add_columns<64>(v, u, k);
                    tmem_ld_32x32b_x32(lanes, t);
                    add_columns<0>(v, t, k);
                }
                ++use;
                if (c0 + CHUNK >= k.kt1) break;
            }
            if (!ok) {
                atomicOr(P.err, ERR_TIMEOUT_ACC);
                *abort_flag = 1;
                break;
            }
            if (k.piece) {
                // The piece to memory; whoever brings the last piece of this warp's part of a tile adds them up in
                // their order.  (Part by part: no warp waits for another one, which may have given up.)
                const long long slot = (long long)TILE * TILE;
                const long long part = (long long)rank * HALF * TILE + e * (32 * COLS) + lane * 4;
                float *mine = P.partial + (2 * pair + (k.kt0 == 0)) * slot + part;
#pragma unroll
                for (int c = 0; c < COLS; c += 4)
                    *(float4 *)(mine + c * 32) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                __threadfence();
                const Pieces pieces = pieces_of(P, k.begin, q.k_tiles, pair);
                const int first = pieces.first, last = pieces.last;
                __syncwarp();
                int there = 0;
                if (lane == 0) there = atomicAdd(&P.counters[(2 * first + rank) * EPI_WARPS + e], 1) + 1;
                if (__shfl_sync(0xffffffffu, there, 0) != pieces.count) continue;
                __syncwarp();
                __threadfence();
#pragma unroll
                for (int c = 0; c < COLS; c += 64) {
#pragma unroll
                    for (int i = 0; i < 64; ++i) v[c + i] = 0.f;
#pragma unroll 1
                    for (int s = first; s <= last; ++s) {
                        if (s > first && P.share[s] == P.share[s - 1]) continue;  // (an empty share)
                        const float *from = P.partial + (2 * s + (s == first)) * slot + part + c * 32;
                        float4 f[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = __ldcg((const float4 *)(from + i * 128));
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            v[c + 4 * i] += f[i].x;
                            v[c + 4 * i + 1] += f[i].y;
                            v[c + 4 * i + 2] += f[i].z;
                            v[c + 4 * i + 3] += f[i].w;
                        }
                    }
                }
            }
            // (one copy of the stores' code for all chunks: what it costs is mostly fetching it)
#pragma unroll 1
            for (int c = 0; c < COLS; c += 32) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *(float4 *)(stage + lane * LD + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                __syncwarp();
                bad |= store_chunk(q, i0, j0 + 2 * c, stage, lane);
                __syncwarp();
#pragma unroll
                for (int i = 0; i + 32 < COLS; ++i) v[i] = v[i + 32];
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(P.err, ERR_NONFINITE);
    }
    __syncthreads();
    cluster_sync();  // nothing of either CTA is used by the other any more
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem);
    }
}

// The error word and the counters of a call.  A kernel, not a memset: the next kernel's start
// overlaps it.
__global__ void zero_kernel(int *err, int *counters, int n) {
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x == 0 && err) *err = 0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) counters[i] = 0;
}

// ------------------------------------------------------------------ host

bool element_map(CUtensorMap *m, const void *q, long long ld, long long rows, int width) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128u, (cuuint32_t)BK}, step[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)q, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Tiles of 512 bytes of exponents.
bool exponent_map(CUtensorMap *m, const void *s, long long tiles) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {128u, (cuuint64_t)tiles}, strides[1] = {512u};
    const cuuint32_t box[2] = {128u, 1u}, step[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, (void *)s, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs that run at the same time on the current device.  Asked once for each device, where
// the kernels' shared memory is allowed first.
int pairs() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaFuncSetAttribute(mx_kernel<FEW_PROBS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
        cudaFuncSetAttribute(mx_kernel<MAX_PROBS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * device_sm_count());
        cfg.blockDim = dim3(NUM_THREADS);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, mx_kernel<FEW_PROBS>, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = std::max(1, device_sm_count() / 2);
        }
        cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

Tiles tiles_of(const MxJob &j) {
    return Tiles{(int)ceil_div(j.M, TILE), (int)ceil_div(j.N, TILE), (int)ceil_div(j.K, BK), j.sym != 0, 0, 0};
}

// The launches of a call, and the scratch that they share (they follow one another).
struct Plan {
    std::vector<int> order;
    std::vector<Launch> launches;
    float *partial = nullptr;
    int *counters = nullptr;
    size_t ncounters = 0;
};

size_t counters_of(const Launch &l) { return (size_t)l.pairs * 2 * EPI_WARPS; }

Plan make_plan(const MxJob *jobs, int n, Arena &ws) {
    Plan p;
    p.order.resize(n);
    for (int i = 0; i < n; ++i) p.order[i] = i;
    std::stable_sort(p.order.begin(), p.order.end(), [&](int x, int y) { return jobs[x].K > jobs[y].K; });
    std::vector<Tiles> tiles(n);
    for (int i = 0; i < n; ++i) tiles[i] = tiles_of(jobs[p.order[i]]);
    const int most = std::min(pairs(), MAX_PAIRS);
    int slots = 0;
    for (int at = 0; at < n; at = p.launches.back().to) {
        p.launches.push_back(make_launch(tiles, at, most));
        if (const Launch &l = p.launches.back(); l.span > 0) {
            slots = std::max(slots, 2 * l.pairs);
            p.ncounters += counters_of(l);
        }
    }
    p.counters = ws.take<int>(std::max<size_t>(p.ncounters, 1));
    p.partial = ws.take<float>((size_t)slots * TILE * TILE);
    return p;
}

}  // namespace

size_t mx_workspace_bytes(const MxJob *jobs, int njobs) {
    if (njobs <= 0) return 0;
    Arena a;
    make_plan(jobs, njobs, a);
    return a.used;
}

namespace {

template <int CAP>
kfac_status launch(const MxJob *jobs, const Plan &p, const Launch &l, int *counters, int *err, bool alone, cudaStream_t st) {
    std::unique_ptr<Params<CAP>> P(new Params<CAP>());
    static_cast<Deal &>(*P) = l.deal;
    P->partial = p.partial;
    P->counters = counters;
    P->err = err;
    P->alone = alone;
    for (int i = 0; i < P->nprob; ++i) {
        const MxJob &j = jobs[p.order[l.from + i]];
        Prob &q = P->prob[i];
        static_cast<Tiles &>(q) = l.tiles[i];
        const long long sa_tiles = ceil_div(j.M, HALF) * q.k_tiles, sb_tiles = ceil_div(j.N, HALF) * q.k_tiles;
        if (j.K > 0) {  // (without rows nothing is loaded)
            if (!element_map(&q.a, j.a, j.lda, j.K, j.M) || !exponent_map(&q.sa, j.sa, sa_tiles)) return KFAC_ERR_CUDA;
            if (j.sym) {
                q.b = q.a;
                q.sb = q.sa;
            } else if (!element_map(&q.b, j.b, j.ldb, j.K, j.N) || !exponent_map(&q.sb, j.sb, sb_tiles)) {
                return KFAC_ERR_CUDA;
            }
        }
        q.C = j.C;
        q.ldc = j.ldc;
        q.M = j.M;
        q.N = j.N;
        q.alpha = j.alpha;
        q.beta = j.beta;
        q.packed = j.packed != 0;
        q.c_dtype = (uint8_t)j.c_dtype;
        q.vec = !j.packed && j.ldc % 4 == 0 && (uintptr_t)j.C % (j.c_dtype == KFAC_F32 ? 16 : 8) == 0;
    }
    KFAC_LAUNCH_CLUSTERS(KK_MX, st, mx_kernel<CAP>, 2, 2 * l.pairs, NUM_THREADS, SMEM_BYTES, *P);
    return KFAC_OK;
}

kfac_status run_plan(const MxJob *jobs, const Plan &p, int *err, bool zero_err, cudaStream_t st) {
    // (one pair of CTAs sets the error word to 0 itself)
    const bool alone = zero_err && p.launches.size() == 1 && p.launches[0].pairs == 1 && !p.ncounters;
    if (!alone && (zero_err || p.ncounters))
        KFAC_LAUNCH(KK_MX, st, zero_kernel, 1, 256, 0, zero_err ? err : nullptr, p.counters, (int)p.ncounters);
    int *counters = p.counters;
    for (const Launch &l : p.launches) {
        const kfac_status s = l.deal.nprob <= FEW_PROBS ? launch<FEW_PROBS>(jobs, p, l, counters, err, alone, st)
                                                        : launch<MAX_PROBS>(jobs, p, l, counters, err, alone, st);
        if (s != KFAC_OK) return s;
        if (l.span > 0) counters += counters_of(l);
    }
    return KFAC_OK;
}

}  // namespace

kfac_status mx_run(const MxJob *jobs, int njobs, Arena &ws, int *err, bool zero_err, cudaStream_t st) {
    if (njobs <= 0) return KFAC_OK;
    const Plan p = make_plan(jobs, njobs, ws);
    return ws.fits() ? run_plan(jobs, p, err, zero_err, st) : KFAC_ERR_WORKSPACE;
}

namespace {

kfac_status check_weight_grad(const kfac_weight_grad_desc *descs, int count, std::vector<MxJob> &jobs) {
    if (count < 0 || (count > 0 && !descs)) return KFAC_ERR_INVALID;
    for (int i = 0; i < count; ++i) {
        const kfac_weight_grad_desc &d = descs[i];
        if (d.out_dtype != KFAC_F32 && d.out_dtype != KFAC_BF16 && d.out_dtype != KFAC_F16) return KFAC_ERR_INVALID;
        if (d.dA < 1 || d.dG < 1 || !d.out || d.ld < d.dA || (uintptr_t)d.out % (d.out_dtype == KFAC_F32 ? 4 : 2) ||
            !std::isfinite(d.alpha) || !std::isfinite(d.beta))
            return KFAC_ERR_INVALID;
        kfac_status s = check_checkpoint(d.q_a, d.ldq_a, d.scales_a, d.rows, d.dA);
        if (s == KFAC_OK) s = check_checkpoint(d.q_g, d.ldq_g, d.scales_g, d.rows, d.dG);
        if (s != KFAC_OK) return s;
        jobs.push_back(MxJob{d.q_g, d.ldq_g, d.scales_g, d.q_a, d.ldq_a, d.scales_a, d.rows, d.dG, d.dA, 0, 0, d.out,
                             d.ld, d.out_dtype, d.alpha, d.beta});
    }
    return KFAC_OK;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" size_t kfac_weight_grad_workspace_size(const kfac_weight_grad_desc *descs, int count) {
    std::vector<MxJob> jobs;
    if (check_weight_grad(descs, count, jobs) != KFAC_OK) return 0;
    Arena a;
    a.take<int>(64);  // the error word
    make_plan(jobs.data(), count, a);
    return a.used;
}

extern "C" kfac_status kfac_weight_grad(const kfac_weight_grad_desc *descs, int count, void *workspace,
                                        size_t workspace_bytes, void *stream) {
    std::vector<MxJob> jobs;
    kfac_status s = check_weight_grad(descs, count, jobs);
    if (s != KFAC_OK || count == 0) return s;
    if (!workspace || ((uintptr_t)workspace % 256) != 0) return KFAC_ERR_WORKSPACE;
    Arena ws(workspace, workspace_bytes);
    int *err = ws.take<int>(64);
    const Plan p = make_plan(jobs.data(), count, ws);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    DeviceMemory memory;
    for (const kfac_weight_grad_desc *d = descs; d < descs + count; ++d)
        if (!memory.holds(d->out, 0) || (d->rows > 0 && !(memory.holds(d->q_a, 1) && memory.holds(d->scales_a, 2) &&
                                                          memory.holds(d->q_g, 1) && memory.holds(d->scales_g, 2))))
            return KFAC_ERR_INVALID;
    return run_plan(jobs.data(), p, err, true, (cudaStream_t)stream);
}
