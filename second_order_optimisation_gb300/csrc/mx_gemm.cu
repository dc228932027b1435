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
// A persistent kernel of ten warps: one brings operand tiles by TMA, one thread issues the
// products, and eight take the accumulator out of tensor memory into registers at once,
// so that the next tile's products start before this one's stores.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <mutex>
#include <vector>

#include "internal.h"

namespace kfac {
namespace {

constexpr int BM = 128, BN = 128, BK = 128;  // a CTA's tile: features x features, tokens a stage
constexpr int STAGES = 5;
constexpr int TILE_BYTES = 128 * 128, SF_BYTES = 512;
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int SF_STAGE = 2 * SF_BYTES;
constexpr int EPI_WARPS = 8, NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int COLS = BN / 2;  // accumulator columns of an epilogue warp
constexpr int LD = 33;        // pitch of its staging chunk
constexpr int SF_COL = 256, SF_SLOT = 16;  // tensor memory: exponents, a slot for each stage
constexpr int TMEM_COLS = 512;
constexpr int MAX_PROBS = 48, GROUP = 8;
constexpr int CHUNK = 16;  // stages (2048 tokens) in one accumulator
constexpr size_t SMEM_BYTES =
    1024 + STAGES * (STAGE_BYTES + SF_STAGE) + EPI_WARPS * 32 * LD * sizeof(float) + 256;

struct Prob {
    CUtensorMap a, b, sa, sb;
    void *C;
    float *partial;
    int *counters;
    long long ldc;
    int M, N, k_tiles, tiles_m, tiles_n, ksplit, work_begin;
    float alpha, beta;
    uint8_t sym, packed, c_dtype;
};
struct Params {
    Prob prob[MAX_PROBS];
    int nprob, total_work;
    int *err;
};
static_assert(sizeof(Params) <= 32000, "kernel parameters");

struct Work {
    int p, tm, tn, tile, split, kt0, kt1;
};

__device__ __forceinline__ Work decode(const Params &P, int w) {
    int lo = 0, hi = P.nprob - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.prob[mid].work_begin <= w) lo = mid;
        else hi = mid - 1;
    }
    const Prob &q = P.prob[lo];
    Work k;
    k.p = lo;
    const int local = w - q.work_begin;
    k.tile = local / q.ksplit;
    k.split = local - k.tile * q.ksplit;
    // bands of GROUP rows of tiles, column by column, so that the CTAs at work together
    // share panels of both operands in L2; of a symmetric result the upper tiles
    const int T = q.tiles_n;
    int u = k.tile;
    if (q.sym) {
        int b0 = 0, gb;
        for (;;) {
            gb = min(GROUP, T - b0);
            const int size = gb * (T - b0) - gb * (gb - 1) / 2;
            if (u < size) break;
            u -= size;
            b0 += gb;
        }
        const int stair = gb * (gb + 1) / 2;
        if (u < stair) {
            int c = 0;
            while (u > c) u -= ++c;
            k.tn = b0 + c;
            k.tm = b0 + u;
        } else {
            u -= stair;
            k.tn = b0 + gb + u / gb;
            k.tm = b0 + u % gb;
        }
    } else {
        const int band = u / (GROUP * T), b0 = band * GROUP, gb = min(GROUP, q.tiles_m - b0);
        u -= b0 * T;
        k.tn = u / gb;
        k.tm = b0 + u % gb;
    }
    k.kt0 = (int)((long long)k.split * q.k_tiles / q.ksplit);
    k.kt1 = (int)((long long)(k.split + 1) * q.k_tiles / q.ksplit);
    return k;
}

// Shared-memory descriptor of a slice of 32 tokens: groups of 8 rows of 128 features,
// 128-byte swizzle, 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t tile, int slice) {
    return smem_desc_sw128(tile + slice * 4096, TILE_BYTES, 1024);
}
// Of 512 bytes of exponents: 32 rows of 16 bytes, groups of 8 rows 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t exponents(uint32_t at) {
    return (uint64_t)((at & 0x3FFFF) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// Copies them to four columns of tensor memory, the same for each quarter of the lanes.
__device__ __forceinline__ void copy_exponents(uint32_t tmem, uint32_t smem) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(exponents(smem)) : "memory");
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
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float old_value(const Prob &q, long long at) {
    if (q.c_dtype == KFAC_F32) return ((const float *)q.C)[at];
    const uint16_t b = ((const uint16_t *)q.C)[at];
    return q.c_dtype == KFAC_F16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_f32(b);
}

// Stores 32 rows x 32 columns at (i0, j0): v is a row to a lane; through the warp's
// stage, so that a lane then has a column and every access of a warp is one run of a row, at
// any pitch or packing.  Returns whether a value was NaN or infinite.
__device__ __forceinline__ bool store_chunk(const Prob &q, int i0, int j0, const float *v, float *stage, int lane) {
#pragma unroll
    for (int c = 0; c < 32; ++c) stage[lane * LD + c] = v[c];
    __syncwarp();
    const int rows = min(32, q.M - i0), j = j0 + lane;
    bool bad = false;
    if (j0 < q.N && (!q.sym || j0 + 31 >= i0)) {
        const bool in = j < q.N;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 8) {
            float old[8];
            long long at[8];
            bool is[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int i = i0 + r0 + r;
                is[r] = in && r0 + r < rows && (!q.sym || j >= i);
                at[r] = (q.packed ? (long long)i * q.N - (long long)i * (i + 1) / 2 : (long long)i * q.ldc) + j;
                old[r] = q.beta != 0.f && is[r] ? old_value(q, at[r]) : 0.f;
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (!is[r]) continue;
                const float x = fmaf(q.beta, old[r], q.alpha * stage[(r0 + r) * LD + lane]);
                bad |= !(fabsf(x) <= 3.402823466e38f);
                if (q.c_dtype == KFAC_F32) ((float *)q.C)[at[r]] = x;
                else ((uint16_t *)q.C)[at[r]] = f32_to_16_bits(x, q.c_dtype == KFAC_F16);
            }
        }
    }
    __syncwarp();
    return bad;
}

__global__ void __launch_bounds__(NUM_THREADS, 1) mx_kernel(const __grid_constant__ Params P) {
    extern __shared__ uint8_t raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sf = smem + STAGES * STAGE_BYTES;
    float *stages = (float *)(sf + STAGES * SF_STAGE);
    uint64_t *full = (uint64_t *)(stages + EPI_WARPS * 32 * LD);
    uint64_t *empty = full + STAGES;
    uint64_t *accf = empty + STAGES, *acce = accf + 1, *drain = acce + 1;
    uint32_t *tmem_slot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tmem_slot + 1);
    volatile int *last_flag = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accf, 1);
        mbar_init(acce, EPI_WARPS);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int w = blockIdx.x; w < P.total_work && !*abort_flag; w += gridDim.x) {
                const Work k = decode(P, w);
                const Prob &q = P.prob[k.p];
                const bool same = q.sym && k.tm == k.tn;
                for (int kt = k.kt0; kt < k.kt1 && !*abort_flag; ++kt) {
                    if (!mbar_wait(&empty[stage], phase ^ 1)) {
                        atomicOr(P.err, ERR_TIMEOUT_EMPTY);
                        *abort_flag = 1;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[stage], (same ? 1 : 2) * (TILE_BYTES + SF_BYTES));
                    uint8_t *s = smem + stage * STAGE_BYTES, *f = sf + stage * SF_STAGE;
                    tma_load_2d(s, &q.a, k.tm * BM, kt * BK, &full[stage]);
                    tma_load_2d(f, &q.sa, 0, k.tm * q.k_tiles + kt, &full[stage]);
                    if (!same) {
                        tma_load_2d(s + TILE_BYTES, &q.b, k.tn * BN, kt * BK, &full[stage]);
                        tma_load_2d(f + SF_BYTES, &q.sb, 0, k.tn * q.k_tiles + kt, &full[stage]);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    ++issued;
                }
            }
            if (*abort_flag) {  // cut short: the copies that are on their way land before the CTA leaves
                for (int n = 0; n < min(issued, STAGES); ++n) {
                    if (stage == 0) { stage = STAGES - 1; phase ^= 1; } else { --stage; }
                    if (!mbar_wait(&full[stage], phase)) atomicOr(P.err, ERR_TIMEOUT_DRAIN);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, use = 0;
            bool ok = true;
            for (int w = blockIdx.x; w < P.total_work && ok && !*abort_flag; w += gridDim.x) {
                const Work k = decode(P, w);
                const Prob &q = P.prob[k.p];
                const bool same = q.sym && k.tm == k.tn;
                for (int c0 = k.kt0; ok; c0 += CHUNK) {
                    const int c1 = min(k.kt1, c0 + CHUNK);
                    if (!mbar_wait(acce, (use & 1) ^ 1)) {
                        atomicOr(P.err, ERR_TIMEOUT_ACC);
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    ++use;
                    tc_fence_after();
                    for (int kt = c0; kt < c1; ++kt) {
                        if (!mbar_wait(&full[stage], phase)) {
                            atomicOr(P.err, ERR_TIMEOUT_FULL);
                            *abort_flag = 1;
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a = smem_u32(smem + stage * STAGE_BYTES), b = same ? a : a + TILE_BYTES;
                        const uint32_t f = smem_u32(sf + stage * SF_STAGE);
                        const uint32_t ta = tmem + SF_COL + stage * SF_SLOT, tb = ta + 4;
                        // (a slot of exponents is written again when its stage's products are done)
                        copy_exponents(ta, f);
                        copy_exponents(tb, same ? f : f + SF_BYTES);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma(tmem, operand(a, s), operand(b, s), idesc(BM, BN, s), ta, tb, kt > c0 || s > 0);
                        tc_commit(&empty[stage]);
                        if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    tc_commit(accf);
                    if (c1 >= k.kt1) break;
                }
            }
            if (*abort_flag) {
                tc_commit(drain);
                if (!mbar_wait(drain, 0)) atomicOr(P.err, ERR_TIMEOUT_DRAIN);
            }
        }
    } else {
        const int e = warp - 2, quarter = warp & 3, half = e >> 2;
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + half * COLS;
        float *stage = stages + e * 32 * LD;
        uint32_t use = 0;
        bool bad = false;
        for (int w = blockIdx.x; w < P.total_work && !*abort_flag; w += gridDim.x) {
            const Work k = decode(P, w);
            const Prob &q = P.prob[k.p];
            float v[COLS];
            bool ok = true;
            for (int c0 = k.kt0;; c0 += CHUNK) {
                if (!mbar_wait(accf, use & 1)) {
                    ok = false;
                    break;
                }
                ++use;
                tc_fence_after();
                // (without a token nothing was multiplied: the accumulator holds another tile's values)
                const bool first = c0 == k.kt0, none = k.kt0 >= k.kt1;
#pragma unroll
                for (int c = 0; c < COLS; c += 32) {
                    float t[32];
                    tmem_ld_32x32b_x32(at + c, t);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[c + i] = none ? 0.f : first ? t[i] : v[c + i] + t[i];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce);
                if (c0 + CHUNK >= k.kt1) break;
            }
            if (!ok) {
                atomicOr(P.err, ERR_TIMEOUT_ACC);
                *abort_flag = 1;
                break;
            }
            const int i0 = k.tm * BM + quarter * 32, j0 = k.tn * BN + half * COLS;
            if (q.ksplit > 1) {
                const long long span = (long long)BM * BN;
                float *mine = q.partial + ((long long)k.tile * q.ksplit + k.split) * span + e * (32 * COLS) + lane;
#pragma unroll
                for (int c = 0; c < COLS; ++c) mine[c * 32] = v[c];
                __threadfence();
                named_barrier_sync(1, 32 * EPI_WARPS);
                if (threadIdx.x == 64) *last_flag = atomicAdd(&q.counters[k.tile], 1) == q.ksplit - 1;
                named_barrier_sync(1, 32 * EPI_WARPS);
                const bool last = *last_flag != 0;
                named_barrier_sync(1, 32 * EPI_WARPS);
                if (!last) continue;
                __threadfence();
                const float *all = q.partial + (long long)k.tile * q.ksplit * span + e * (32 * COLS) + lane;
#pragma unroll
                for (int c = 0; c < COLS; ++c) v[c] = __ldcg(all + c * 32);
                for (int s = 1; s < q.ksplit; ++s) {
#pragma unroll
                    for (int c = 0; c < COLS; ++c) v[c] += __ldcg(all + s * span + c * 32);
                }
            }
#pragma unroll
            for (int c = 0; c < COLS; c += 32) bad |= store_chunk(q, i0, j0 + c, v + c, stage, lane);
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(P.err, ERR_NONFINITE);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
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

struct Plan {
    std::vector<int> tiles, ksplit, k_tiles;
    std::vector<float *> partial;
    std::vector<int *> counters;
    int *counter_base = nullptr;
    size_t ncounters = 0;
};

int tiles_of(const MxJob &j) {
    const int tm = (int)ceil_div(j.M, BM), tn = (int)ceil_div(j.N, BN);
    return j.sym ? tm * (tm + 1) / 2 : tm * tn;
}

Plan make_plan(const MxJob *jobs, int n, Arena &ws) {
    Plan p;
    double total = 0;
    for (int i = 0; i < n; ++i) {
        p.tiles.push_back(tiles_of(jobs[i]));
        p.k_tiles.push_back((int)ceil_div(jobs[i].K, BK));
        total += (double)p.tiles[i] * p.k_tiles[i];
    }
    // a tile's tokens are split where it would be the critical path: no item of more than
    // about half of an SM's share, none of fewer than 8 stages
    const double target = std::max(8.0, total / (2.0 * device_sm_count()));
    for (int i = 0; i < n; ++i) {
        const int ks = (int)std::min(64.0, std::ceil(p.k_tiles[i] / target));
        p.ksplit.push_back(std::max(1, ks));
        if (p.ksplit[i] > 1) p.ncounters += p.tiles[i];
    }
    p.counter_base = ws.take<int>(std::max<size_t>(p.ncounters, 1));
    size_t at = 0;
    for (int i = 0; i < n; ++i) {
        const bool split = p.ksplit[i] > 1;
        p.partial.push_back(split ? ws.take<float>((size_t)p.tiles[i] * p.ksplit[i] * BM * BN) : nullptr);
        p.counters.push_back(split && p.counter_base ? p.counter_base + at : nullptr);
        if (split) at += p.tiles[i];
    }
    return p;
}

}  // namespace

size_t mx_workspace_bytes(const MxJob *jobs, int njobs) {
    if (njobs <= 0) return 0;
    Arena a;
    make_plan(jobs, njobs, a);
    return a.used;
}

kfac_status mx_run(const MxJob *jobs, int njobs, Arena &ws, int *err, cudaStream_t st) {
    if (njobs <= 0) return KFAC_OK;
    static std::once_flag once;
    static cudaError_t attr = cudaSuccess;
    std::call_once(once, [] {
        attr = cudaFuncSetAttribute(mx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    });
    if (attr != cudaSuccess) return KFAC_ERR_CUDA;
    const Plan p = make_plan(jobs, njobs, ws);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    if (p.ncounters) KFAC_CUDA_TRY(cudaMemsetAsync(p.counter_base, 0, p.ncounters * sizeof(int), st));
    std::vector<int> order(njobs);  // long items first
    for (int i = 0; i < njobs; ++i) order[i] = i;
    std::stable_sort(order.begin(), order.end(), [&](int x, int y) {
        return (long long)p.k_tiles[x] * p.ksplit[y] > (long long)p.k_tiles[y] * p.ksplit[x];
    });
    std::unique_ptr<Params> P(new Params);
    for (int at = 0; at < njobs;) {
        P->nprob = P->total_work = 0;
        for (; at < njobs && P->nprob < MAX_PROBS; ++at) {
            const MxJob &j = jobs[order[at]];
            const int i = order[at];
            if ((long long)P->total_work + (long long)p.tiles[i] * p.ksplit[i] > 0x7fffffffLL) break;
            Prob &q = P->prob[P->nprob++];
            std::memset(&q, 0, sizeof(q));
            q.k_tiles = p.k_tiles[i];
            q.tiles_m = (int)ceil_div(j.M, BM);
            q.tiles_n = (int)ceil_div(j.N, BN);
            if (j.K > 0) {  // (without rows nothing is loaded)
                if (!element_map(&q.a, j.a, j.lda, j.K, j.M) || !exponent_map(&q.sa, j.sa, (long long)q.tiles_m * q.k_tiles))
                    return KFAC_ERR_CUDA;
                if (j.sym) {
                    q.b = q.a;
                    q.sb = q.sa;
                } else if (!element_map(&q.b, j.b, j.ldb, j.K, j.N) ||
                           !exponent_map(&q.sb, j.sb, (long long)q.tiles_n * q.k_tiles)) {
                    return KFAC_ERR_CUDA;
                }
            }
            q.C = j.C;
            q.ldc = j.ldc;
            q.partial = p.partial[i];
            q.counters = p.counters[i];
            q.M = j.M;
            q.N = j.N;
            q.ksplit = p.ksplit[i];
            q.work_begin = P->total_work;
            q.alpha = j.alpha;
            q.beta = j.beta;
            q.sym = j.sym != 0;
            q.packed = j.packed != 0;
            q.c_dtype = (uint8_t)j.c_dtype;
            P->total_work += p.tiles[i] * p.ksplit[i];
        }
        P->err = err;
        const int grid = std::max(1, std::min(P->total_work, device_sm_count()));
        KFAC_LAUNCH(KK_MX, st, mx_kernel, grid, NUM_THREADS, SMEM_BYTES, *P);
    }
    return KFAC_OK;
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
    Arena ws(workspace, workspace_bytes), probe(workspace, workspace_bytes);
    probe.take<int>(64);
    make_plan(jobs.data(), count, probe);
    if (!probe.fits()) return KFAC_ERR_WORKSPACE;
    for (const kfac_weight_grad_desc *d = descs; d < descs + count; ++d)
        if (!all_on_this_device({d->out}) ||
            (d->rows > 0 && !all_on_this_device({d->q_a, d->scales_a, d->q_g, d->scales_g})))
            return KFAC_ERR_INVALID;
    int *err = ws.take<int>(64);
    cudaStream_t st = (cudaStream_t)stream;
    KFAC_CUDA_TRY(cudaMemsetAsync(err, 0, sizeof(int), st));
    return mx_run(jobs.data(), count, ws, err, st);
}
