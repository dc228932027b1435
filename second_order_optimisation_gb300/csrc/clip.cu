// clip.cu -- kfac_clip_norm: the norm over many tensors, clipping, and the
// step on the weights.
//
//   norm = sqrt(sum x y)  (y = x: the Euclidean norm),  scale = min(1, max_norm / norm),
//   out = scale x,  w <- w - eta scale x.
//
// Two passes over a list of chunks: every CTA sums its chunks' products (fp32
// in the threads, fp64 across them and across chunks, in a fixed order), then
// every chunk is scaled.  A chunk whose fp32 sum overflows or vanishes is
// summed again from values scaled by a power of two, so that any finite input
// gives its norm.
#include <algorithm>
#include <cmath>
#include <memory>

#include "logits.cuh"

namespace kfac {
namespace {

constexpr int CLIP_MAX = 256;      // tensors of one launch (kernel parameters)
constexpr int CLIP_THREADS = 256;
constexpr int CHUNK = 8192;        // elements of a chunk

struct ClipJob {
    const char *x, *y;
    char *out;
    float *w;
    long long ld, ld_y, ld_out, ld_w;
    long long rows, cols;  // a tensor without gaps is one row
    int dtype, out_dtype;
    int per_row;           // chunks of a row
    int first;             // index of its first chunk in the launch
};
struct ClipParams {
    ClipJob job[CLIP_MAX];
    int n, chunks;
    int part0;             // where this launch's partial sums start
    double *part;          // one for each chunk
    const float *scale;
    float eta;
};

template <int DT>
__device__ __forceinline__ float elem(const char *p, long long i) {
    return Elem<DT>::value(((const typename Elem<DT>::bits *)p)[i]);
}
__device__ __forceinline__ float elem(int dt, const char *p, long long i) {
    return dt == KFAC_BF16 ? elem<KFAC_BF16>(p, i) : dt == KFAC_F16 ? elem<KFAC_F16>(p, i) : elem<KFAC_F32>(p, i);
}

__device__ __forceinline__ const ClipJob &job_of(const ClipParams &P, int chunk) {
    int lo = 0, hi = P.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.job[mid].first <= chunk) lo = mid; else hi = mid - 1;
    }
    return P.job[lo];
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[CLIP_THREADS / 32];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    double all = 0;
    for (int i = 0; i < CLIP_THREADS / 32; ++i) all += part[i];
    return all;
}
__device__ __forceinline__ unsigned block_max(unsigned v) {
    __shared__ unsigned part[CLIP_THREADS / 32];
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    unsigned all = 0;
    for (int i = 0; i < CLIP_THREADS / 32; ++i) all = max(all, part[i]);
    return all;
}

// 2^n as fp32, n in -126 .. 127.
__device__ __forceinline__ float pow2(int n) { return __int_as_float((n + 127) << 23); }
// A power of two (as its exponent) that brings the largest magnitude (its bits) near 1.
__device__ __forceinline__ int to_one(unsigned magnitude) {
    return max(-126, min(126, 127 - (int)(magnitude >> 23)));
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_norm_kernel(const __grid_constant__ ClipParams P) {
    pdl_wait();
    pdl_trigger();
    const int chunk = blockIdx.x;
    const ClipJob &j = job_of(P, chunk);
    const int rel = chunk - j.first;
    const long long row = rel / j.per_row, c0 = (long long)(rel % j.per_row) * CHUNK;
    const int n = (int)min((long long)CHUNK, j.cols - c0);
    const int es = j.dtype == KFAC_F32 ? 4 : 2;
    const char *x = j.x + (row * j.ld + c0) * es, *y = j.y ? j.y + (row * j.ld_y + c0) * es : x;
    float s = 0.f;
    for (int i = threadIdx.x; i < n; i += CLIP_THREADS) s = fmaf(elem(j.dtype, x, i), elem(j.dtype, y, i), s);
    double all = block_sum((double)s);
    // squares overflow from 2^64 and lose bits below 2^-63
    if (!(fabs(all) <= (double)F32_MAX) || fabs(all) < 1e-28) {
        unsigned mx = 0, my = 0;
        for (int i = threadIdx.x; i < n; i += CLIP_THREADS) {
            mx = max(mx, __float_as_uint(elem(j.dtype, x, i)) & 0x7fffffffu);
            my = max(my, __float_as_uint(elem(j.dtype, y, i)) & 0x7fffffffu);
        }
        mx = block_max(mx);
        my = block_max(my);
        if (mx < 0x7f800000u && my < 0x7f800000u) {
            const int ex = to_one(mx), ey = to_one(my);
            s = 0.f;
            for (int i = threadIdx.x; i < n; i += CLIP_THREADS)
                s = fmaf(elem(j.dtype, x, i) * pow2(ex), elem(j.dtype, y, i) * pow2(ey), s);
            all = ldexp(block_sum((double)s), -ex - ey);
        }
    }
    if (threadIdx.x == 0) P.part[P.part0 + chunk] = all;
}

struct ClipTotal {
    const double *part;
    long long n;
    float max_norm;
    float *norm, *scale_out, *scale;
    int *err;
};
__global__ void __launch_bounds__(CLIP_THREADS) clip_total_kernel(const ClipTotal P) {
    pdl_wait();
    pdl_trigger();
    double s = 0;
    for (long long i = threadIdx.x; i < P.n; i += CLIP_THREADS) s += P.part[i];
    s = block_sum(s);
    if (threadIdx.x == 0) {
        const float norm = (float)sqrt(s < 0 ? 0. : s);
        const float scale = norm > P.max_norm ? P.max_norm / norm : norm <= P.max_norm ? 1.f : norm;
        *P.scale = scale;
        if (P.norm) *P.norm = norm;
        if (P.scale_out) *P.scale_out = scale;
        *P.err = finite(norm) ? 0 : ERR_NONFINITE;
    }
}

template <int DT>
__device__ __forceinline__ void put(char *p, long long i, float v) {
    ((typename Elem<DT>::bits *)p)[i] = Elem<DT>::round(v);
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_apply_kernel(const __grid_constant__ ClipParams P) {
    pdl_wait();
    pdl_trigger();
    const int chunk = blockIdx.x;
    const ClipJob &j = job_of(P, chunk);
    const float scale = *P.scale;
    if (!j.w && (!j.out || (j.out == j.x && scale == 1.f))) return;
    const int rel = chunk - j.first;
    const long long row = rel / j.per_row, c0 = (long long)(rel % j.per_row) * CHUNK;
    const int n = (int)min((long long)CHUNK, j.cols - c0);
    const char *x = j.x + (row * j.ld + c0) * (j.dtype == KFAC_F32 ? 4 : 2);
    char *out = j.out ? j.out + (row * j.ld_out + c0) * (j.out_dtype == KFAC_F32 ? 4 : 2) : nullptr;
    float *w = j.w ? j.w + row * j.ld_w + c0 : nullptr;
    for (int i = threadIdx.x; i < n; i += CLIP_THREADS) {
        const float v = scale * elem(j.dtype, x, i);
        if (out) {
            if (j.out_dtype == KFAC_BF16) put<KFAC_BF16>(out, i, v);
            else if (j.out_dtype == KFAC_F16) put<KFAC_F16>(out, i, v);
            else put<KFAC_F32>(out, i, v);
        }
        if (w) w[i] -= P.eta * v;
    }
}

bool known(int dtype) { return dtype == KFAC_BF16 || dtype == KFAC_F16 || dtype == KFAC_F32; }
int size_of(int dtype) { return dtype == KFAC_F32 ? 4 : 2; }

kfac_status check_clip(const kfac_clip_desc *descs, int count, float max_norm, float eta) {
    if (count < 0 || (count > 0 && !descs) || !(max_norm > 0.f) || !std::isfinite(eta)) return KFAC_ERR_INVALID;
    for (int i = 0; i < count; ++i) {
        const kfac_clip_desc &d = descs[i];
        if (d.rows < 0 || d.cols < 0 || !known(d.dtype) || (d.out && !known(d.out_dtype))) return KFAC_ERR_INVALID;
        if (d.rows == 0 || d.cols == 0) continue;
        if (!d.x || d.ld < d.cols || (d.y && d.ld_y < d.cols) || (d.out && d.ld_out < d.cols) ||
            (d.w && d.ld_w < d.cols))
            return KFAC_ERR_INVALID;
        if ((uintptr_t)d.x % size_of(d.dtype) || (uintptr_t)d.y % size_of(d.dtype) ||
            (d.out && (uintptr_t)d.out % size_of(d.out_dtype)) || (uintptr_t)d.w % 4)
            return KFAC_ERR_INVALID;
        if (d.out == d.x && (d.out_dtype != d.dtype || d.ld_out != d.ld)) return KFAC_ERR_INVALID;
    }
    return KFAC_OK;
}

ClipJob job_from(const kfac_clip_desc &d) {
    ClipJob j{(const char *)d.x, (const char *)d.y, (char *)d.out, d.w, d.ld, d.ld_y, d.ld_out, d.ld_w,
              d.rows, d.cols, d.dtype, d.out_dtype, 1, 0};
    if (d.rows == 1 || (d.ld == d.cols && (!d.y || d.ld_y == d.cols) && (!d.out || d.ld_out == d.cols) &&
                        (!d.w || d.ld_w == d.cols))) {
        j.cols = d.rows * d.cols;
        j.rows = 1;
    }
    return j;
}
long long chunks_of(const ClipJob &j) { return j.rows * ceil_div(j.cols, CHUNK); }

long long all_chunks(const kfac_clip_desc *descs, int count) {
    long long n = 0;
    for (int i = 0; i < count; ++i)
        if (descs[i].rows > 0 && descs[i].cols > 0) n += chunks_of(job_from(descs[i]));
    return n;
}

struct ClipPlan {
    int *err;
    float *scale;
    double *part;
};
ClipPlan plan_clip(long long chunks, Arena &ws) {
    ClipPlan p;
    p.err = ws.take<int>(64);
    p.scale = ws.take<float>(1);
    p.part = ws.take<double>((size_t)chunks);
    return p;
}

}  // namespace
}  // namespace kfac

using namespace kfac;

extern "C" size_t kfac_clip_norm_workspace_size(const kfac_clip_desc *descs, int count) {
    if (check_clip(descs, count, 1.f, 0.f) != KFAC_OK) return 0;
    Arena a;
    plan_clip(all_chunks(descs, count), a);
    return a.used;
}

extern "C" kfac_status kfac_clip_norm(const kfac_clip_desc *descs, int count, float max_norm, float eta, float *norm,
                                      float *scale, void *workspace, size_t workspace_bytes, void *stream) {
    kfac_status s = check_clip(descs, count, max_norm, eta);
    if (s != KFAC_OK) return s;
    if (!workspace || ((uintptr_t)workspace % 256) != 0) return KFAC_ERR_WORKSPACE;
    const long long chunks = all_chunks(descs, count);
    if (chunks > 0x7fffffffLL) return KFAC_ERR_UNSUPPORTED;
    Arena ws(workspace, workspace_bytes);
    const ClipPlan p = plan_clip(chunks, ws);
    if (!ws.fits()) return KFAC_ERR_WORKSPACE;
    bool writes = false;
    for (int i = 0; i < count; ++i) {
        const kfac_clip_desc &d = descs[i];
        if (!all_on_this_device({d.x, d.y, d.out, d.w})) return KFAC_ERR_INVALID;
        writes |= d.out || d.w;
    }
    if (!all_on_this_device({norm, scale})) return KFAC_ERR_INVALID;
    cudaStream_t st = (cudaStream_t)stream;
    std::unique_ptr<ClipParams> P(new ClipParams);
    auto pass = [&](bool apply) -> kfac_status {
        int part0 = 0;
        for (int i = 0; i < count;) {
            P->n = P->chunks = 0;
            for (; i < count && P->n < CLIP_MAX; ++i) {
                if (descs[i].rows == 0 || descs[i].cols == 0) continue;
                ClipJob j = job_from(descs[i]);
                j.per_row = (int)ceil_div(j.cols, CHUNK);
                j.first = P->chunks;
                P->chunks += (int)chunks_of(j);
                P->job[P->n++] = j;
            }
            if (P->n == 0) break;
            P->part0 = part0;
            P->part = p.part;
            P->scale = p.scale;
            P->eta = eta;
            part0 += P->chunks;
            if (apply)
                KFAC_LAUNCH(KK_CLIP_APPLY, st, clip_apply_kernel, P->chunks, CLIP_THREADS, 0, *P);
            else
                KFAC_LAUNCH(KK_CLIP_NORM, st, clip_norm_kernel, P->chunks, CLIP_THREADS, 0, *P);
        }
        return KFAC_OK;
    };
    if ((s = pass(false)) != KFAC_OK) return s;
    ClipTotal T{p.part, chunks, max_norm, norm, scale, p.scale, p.err};
    KFAC_LAUNCH(KK_CLIP_NORM, st, clip_total_kernel, 1, CLIP_THREADS, 0, T);
    return writes ? pass(true) : KFAC_OK;
}
