// experts.hip -- rows of a mixture of experts ordered by expert and back.
//
// T tokens choose k experts each: n = T k choices ("slots"), slot t k + j the
// j-th choice of token t.  experts_sort is a stable counting sort of the slots
// by expert; experts_gather writes each token's row to its k places;
// experts_combine adds a token's rows with its weights; experts_combine_backward
// is the gradient of that sum.
#include "gq.h"
#include "gq_internal.h"
#include "matmul.h"

namespace gq {
namespace {

// ---------------------------------------------------------------- sort
// A choice outside 0 .. E - 1 is dropped: it counts as expert E and its place
// is past the last row.  kSortItems slots per workgroup.  The rank of a slot
// among those of its expert is the number before it in its workgroup (by wave
// ballots: the lanes of equal expert are the AND of the ballots of its bits)
// plus the counts of the workgroups before.  No atomics: the order depends on
// nothing but the ids.
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBuckets = GQ_MAX_EXPERTS + 1;

template <typename TI> __device__ inline int bucket_of(const TI *ids, int64_t i, int E)
{
    const TI v = ids[i];
    return v >= 0 && v < (TI)E ? (int)v : E;
}

// Lanes of the wave (of those in `live`) whose bucket is this lane's.
__device__ inline unsigned long long same_bucket(int b, int bits, unsigned long long live)
{
    unsigned long long m = live;
    for (int i = 0; i < bits; ++i) {
        const bool one = (b >> i) & 1;
        const unsigned long long v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

// Counts of each bucket among this workgroup's slots, wave by wave in
// cnt[wave * (E + 1) + bucket] (LDS), and the rank of this thread's slot within
// its wave.  On return cnt holds, for each wave, the number in the waves before.
// Returns the rank within the workgroup; *total (per bucket) to tot.
__device__ inline int rank_in_group(int b, bool in, int E, int bits, unsigned short *cnt, int *tot)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nb = E + 1;
    for (int i = threadIdx.x; i < nb * kSortWaves; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const unsigned long long same = same_bucket(b, bits, __ballot(in));
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (in && rank == 0) cnt[wave * nb + b] = (unsigned short)__popcll(same);
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += kSortThreads) {
        int s = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = cnt[w * nb + i];
            cnt[w * nb + i] = (unsigned short)s;
            s += c;
        }
        tot[i] = s;
    }
    __syncthreads();
    return in ? rank + cnt[wave * nb + b] : 0;
}

// Workgroup w: hist[w (E + 1) + bucket] = its slots of each bucket.
template <typename TI>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(int *hist, const TI *ids, int64_t n, int E)
{
    __shared__ int tot[kMaxBuckets];
    for (int i = threadIdx.x; i <= E; i += kSortThreads) tot[i] = 0;
    __syncthreads();
    const int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
    if (i < n) atomicAdd(&tot[bucket_of(ids, i, E)], 1);      // whole numbers: any order gives the same
    __syncthreads();
    for (int j = threadIdx.x; j <= E; j += kSortThreads) hist[(int64_t)blockIdx.x * (E + 1) + j] = tot[j];
}

// One workgroup: offsets (the exclusive sum of the buckets' totals), and each
// workgroup's count of a bucket replaced by that bucket's first place in it.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(int *hist, int *offsets, int nwg, int E)
{
    __shared__ int base[kMaxBuckets];
    const int nb = E + 1;
    for (int b = threadIdx.x; b < nb; b += kSortThreads) {
        int s = 0;
        for (int w = 0; w < nwg; ++w) s += hist[(int64_t)w * nb + b];
        base[b] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int s = 0;
        for (int b = 0; b < nb; ++b) {
            const int c = base[b];
            base[b] = s;
            offsets[b] = s;                       // offsets[E] = the rows kept
            s += c;
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < nb; b += kSortThreads) {
        int s = base[b];
        for (int w = 0; w < nwg; ++w) {
            const int c = hist[(int64_t)w * nb + b];
            hist[(int64_t)w * nb + b] = s;
            s += c;
        }
    }
}

template <typename TI>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(int *order, int *pos, const int *hist, const TI *ids,
                                                                  int64_t n, int E, int bits)
{
    extern __shared__ unsigned short cnt[];
    __shared__ int tot[kMaxBuckets];
    const int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
    const bool in = i < n;
    const int b = in ? bucket_of(ids, i, E) : E;
    const int rank = rank_in_group(b, in, E, bits, cnt, tot);
    if (!in) return;
    const int p = hist[(int64_t)blockIdx.x * (E + 1) + b] + rank;
    order[p] = b < E ? (int)i : -1;
    pos[i] = b < E ? p : -1;
}

template <typename TI>
hipError_t launch_sort(int *offsets, int *order, int *pos, const TI *ids, int64_t n, int E, int *hist, hipStream_t s)
{
    const int nwg = (int)((n + kSortThreads - 1) / kSortThreads);
    int bits = 0;
    while ((1 << bits) < E + 1) ++bits;
    if (n) hipLaunchKernelGGL(sort_count_kernel<TI>, dim3(nwg), dim3(kSortThreads), 0, s, hist, ids, n, E);
    hipLaunchKernelGGL(sort_scan_kernel, dim3(1), dim3(kSortThreads), 0, s, hist, offsets, nwg, E);
    if (n)
        hipLaunchKernelGGL(sort_place_kernel<TI>, dim3(nwg), dim3(kSortThreads),
                           sizeof(unsigned short) * kSortWaves * (E + 1), s, order, pos, hist, ids, n, E, bits);
    return hipGetLastError();
}

// ---------------------------------------------------------------- gather
constexpr int kRowThreads = 256;

// One token per workgroup: its row read once and written to its k places.
template <typename T, int V>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(T *Xs, int64_t lds, const T *X, int64_t ldx, const int *pos,
                                                             int64_t rows, int64_t Tn, int k, int64_t D)
{
    typedef T vec __attribute__((ext_vector_type(V)));
    const int64_t t = grid_row();
    if (t >= Tn) return;
    const T *x = X + t * ldx;
    for (int64_t c = threadIdx.x * V; c < D; c += kRowThreads * V) {
        const vec v = *(const vec *)(x + c);
        for (int j = 0; j < k; ++j) {
            const int64_t p = pos[t * k + j];
            if (p >= 0 && p < rows) *(vec *)(Xs + p * lds + c) = v;
        }
    }
}

// ---------------------------------------------------------------- combine
template <typename T, int V>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(T *out, int64_t ldo, const T *Y, int64_t ldy,
                                                              const int *pos, const float *w, int64_t rows,
                                                              int64_t Tn, int k, int64_t D)
{
    typedef T vec __attribute__((ext_vector_type(V)));
    const int64_t t = grid_row();
    if (t >= Tn) return;
    for (int64_t c = threadIdx.x * V; c < D; c += kRowThreads * V) {
        float acc[V] = {};
        for (int j = 0; j < k; ++j) {
            const int64_t p = pos[t * k + j];
            if (p < 0 || p >= rows) continue;
            const float wt = w ? w[t * k + j] : 1.0f;
            const vec v = *(const vec *)(Y + p * ldy + c);
#pragma unroll
            for (int u = 0; u < V; ++u) acc[u] = fmaf(wt, (float)v[u], acc[u]);
        }
        vec o;
#pragma unroll
        for (int u = 0; u < V; ++u) o[u] = (T)acc[u];
        *(vec *)(out + t * ldo + c) = o;
    }
}

// One token per workgroup: for each of its rows, dY = w dout and dw = <dout, Y>.
template <typename T, int V>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(T *dY, int64_t lddy, float *dw, const T *dout,
                                                                       int64_t ldo, const T *Y, int64_t ldy,
                                                                       const int *pos, const float *w, int64_t rows,
                                                                       int64_t Tn, int k, int64_t D)
{
    typedef T vec __attribute__((ext_vector_type(V)));
    __shared__ float red[kRowThreads / 64];
    const int64_t t = grid_row();
    if (t >= Tn) return;
    for (int j = 0; j < k; ++j) {
        const int64_t p = pos[t * k + j];
        const bool live = p >= 0 && p < rows;
        const float wt = w[t * k + j];
        float dot = 0.0f;
        if (live)
            for (int64_t c = threadIdx.x * V; c < D; c += kRowThreads * V) {
                const vec g = *(const vec *)(dout + t * ldo + c);
                const vec y = *(const vec *)(Y + p * ldy + c);
                vec o;
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    dot = fmaf((float)g[u], (float)y[u], dot);
                    o[u] = (T)(wt * (float)g[u]);
                }
                *(vec *)(dY + p * lddy + c) = o;
            }
        for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float s = red[0];
            for (int i = 1; i < kRowThreads / 64; ++i) s += red[i];
            dw[t * k + j] = live ? s : 0.0f;
        }
        __syncthreads();
    }
}

// Whether rows of D elements of T at p, ld apart, can be taken in 16-byte pieces.
template <typename T> bool vec_rows(const void *p, int64_t ld, int64_t D)
{
    return ((uintptr_t)p & 15) == 0 && (ld * sizeof(T)) % 16 == 0 && (D * sizeof(T)) % 16 == 0;
}

template <typename T>
hipError_t launch_gather(T *Xs, int64_t lds, const T *X, int64_t ldx, const int *pos, int64_t rows, int64_t Tn, int k,
                         int64_t D, hipStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    const dim3 grid = tile_grid(1, Tn);
    if (vec_rows<T>(Xs, lds, D) && vec_rows<T>(X, ldx, D))
        hipLaunchKernelGGL((gather_kernel<T, V>), grid, dim3(kRowThreads), 0, s, Xs, lds, X, ldx, pos, rows, Tn, k, D);
    else
        hipLaunchKernelGGL((gather_kernel<T, 1>), grid, dim3(kRowThreads), 0, s, Xs, lds, X, ldx, pos, rows, Tn, k, D);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_combine(T *out, int64_t ldo, const T *Y, int64_t ldy, const int *pos, const float *w, int64_t rows,
                          int64_t Tn, int k, int64_t D, hipStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    const dim3 grid = tile_grid(1, Tn);
    if (vec_rows<T>(out, ldo, D) && vec_rows<T>(Y, ldy, D))
        hipLaunchKernelGGL((combine_kernel<T, V>), grid, dim3(kRowThreads), 0, s, out, ldo, Y, ldy, pos, w, rows, Tn, k, D);
    else
        hipLaunchKernelGGL((combine_kernel<T, 1>), grid, dim3(kRowThreads), 0, s, out, ldo, Y, ldy, pos, w, rows, Tn, k, D);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_combine_backward(T *dY, int64_t lddy, float *dw, const T *dout, int64_t ldo, const T *Y, int64_t ldy,
                                   const int *pos, const float *w, int64_t rows, int64_t Tn, int k, int64_t D,
                                   hipStream_t s)
{
    constexpr int V = 16 / sizeof(T);
    const dim3 grid = tile_grid(1, Tn);
    if (vec_rows<T>(dY, lddy, D) && vec_rows<T>(dout, ldo, D) && vec_rows<T>(Y, ldy, D))
        hipLaunchKernelGGL((combine_backward_kernel<T, V>), grid, dim3(kRowThreads), 0, s, dY, lddy, dw, dout, ldo, Y,
                           ldy, pos, w, rows, Tn, k, D);
    else
        hipLaunchKernelGGL((combine_backward_kernel<T, 1>), grid, dim3(kRowThreads), 0, s, dY, lddy, dw, dout, ldo, Y,
                           ldy, pos, w, rows, Tn, k, D);
    return hipGetLastError();
}

int done(hipError_t e)
{
    return e == hipSuccess ? set_error(GQ_OK, "") : set_error(GQ_ERR_HIP, hipGetErrorString(e));
}

// Sizes every call of this file shares; rows is the number of rows of the sorted matrix.
int check_rows(int dtype, int64_t T, int64_t k, int64_t rows, int64_t D)
{
    if (dtype != GQ_F32 && dtype != GQ_BF16) return set_error(GQ_ERR_INVALID_ARG, "unknown dtype");
    if (T < 0 || k < 1 || rows < 0 || D < 1) return set_error(GQ_ERR_INVALID_ARG, "bad sizes");
    if (k > INT32_MAX || T > INT32_MAX / k || rows > INT32_MAX)
        return set_error(GQ_ERR_INVALID_ARG, "size too large");
    return GQ_OK;
}

}  // namespace
}  // namespace gq

using namespace gq;

extern "C" {

size_t experts_sort_workspace_size(int64_t n, int64_t E)
{
    if (n < 0 || n > INT32_MAX || E < 1 || E > GQ_MAX_EXPERTS) return 0;
    return (size_t)((n + kSortThreads - 1) / kSortThreads) * (size_t)(E + 1) * sizeof(int);
}

int experts_sort(int32_t *offsets, int32_t *order, int32_t *pos, const void *ids, int id_bytes, int64_t n, int64_t E,
                 void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (id_bytes != 4 && id_bytes != 8) return set_error(GQ_ERR_INVALID_ARG, "ids must be of 4 or 8 bytes");
    if (n < 0 || n > INT32_MAX) return set_error(GQ_ERR_INVALID_ARG, "bad number of slots");
    if (E < 1 || E > GQ_MAX_EXPERTS) return set_error(GQ_ERR_INVALID_ARG, "E must be 1 .. GQ_MAX_EXPERTS");
    if (!offsets || (n && (!order || !pos || !ids || !ws)))
        return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    if (ws_bytes < experts_sort_workspace_size(n, E)) return set_error(GQ_ERR_INVALID_ARG, "workspace too small");
    return done(id_bytes == 4
                    ? launch_sort(offsets, order, pos, (const int32_t *)ids, n, (int)E, (int *)ws, stream)
                    : launch_sort(offsets, order, pos, (const int64_t *)ids, n, (int)E, (int *)ws, stream));
}

int experts_gather(void *Xs, int64_t ldxs, const void *X, int64_t ldx, int dtype, const int32_t *pos, int64_t rows,
                   int64_t T, int64_t k, int64_t D, hipStream_t stream)
{
    const int rc = check_rows(dtype, T, k, rows, D);
    if (rc) return rc;
    if (ldxs < D || ldx < D) return set_error(GQ_ERR_INVALID_ARG, "a row stride is below the row's length");
    if (T == 0 || rows == 0) return set_error(GQ_OK, "");
    if (!Xs || !X || !pos) return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    return done(dtype == GQ_F32
                    ? launch_gather((float *)Xs, ldxs, (const float *)X, ldx, pos, rows, T, (int)k, D, stream)
                    : launch_gather((__bf16 *)Xs, ldxs, (const __bf16 *)X, ldx, pos, rows, T, (int)k, D, stream));
}

int experts_combine(void *out, int64_t ldo, const void *Y, int64_t ldy, int dtype, const int32_t *pos,
                    const float *weights, int64_t rows, int64_t T, int64_t k, int64_t D, hipStream_t stream)
{
    const int rc = check_rows(dtype, T, k, rows, D);
    if (rc) return rc;
    if (ldo < D || ldy < D) return set_error(GQ_ERR_INVALID_ARG, "a row stride is below the row's length");
    if (T == 0) return set_error(GQ_OK, "");
    if (!out || (rows && !Y) || !pos) return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    return done(dtype == GQ_F32 ? launch_combine((float *)out, ldo, (const float *)Y, ldy, pos, weights, rows, T,
                                                 (int)k, D, stream)
                                : launch_combine((__bf16 *)out, ldo, (const __bf16 *)Y, ldy, pos, weights, rows, T,
                                                 (int)k, D, stream));
}

int experts_combine_backward(void *dY, int64_t lddy, float *dweights, const void *dout, int64_t ldo, const void *Y,
                             int64_t ldy, int dtype, const int32_t *pos, const float *weights, int64_t rows,
                             int64_t T, int64_t k, int64_t D, hipStream_t stream)
{
    const int rc = check_rows(dtype, T, k, rows, D);
    if (rc) return rc;
    if (lddy < D || ldo < D || ldy < D) return set_error(GQ_ERR_INVALID_ARG, "a row stride is below the row's length");
    if (T == 0) return set_error(GQ_OK, "");
    if ((rows && (!dY || !Y)) || !dweights || !dout || !pos || !weights)
        return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    return done(dtype == GQ_F32
                    ? launch_combine_backward((float *)dY, lddy, dweights, (const float *)dout, ldo, (const float *)Y,
                                              ldy, pos, weights, rows, T, (int)k, D, stream)
                    : launch_combine_backward((__bf16 *)dY, lddy, dweights, (const __bf16 *)dout, ldo,
                                              (const __bf16 *)Y, ldy, pos, weights, rows, T, (int)k, D, stream));
}

}  // extern "C"
