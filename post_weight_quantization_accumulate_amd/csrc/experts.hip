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
// A choice outside 0 .. E - 1 is dropped: it counts as expert E, whose places
// come after the last row.  The rank of a slot among those of its expert is the
// number before it in its chunk of 1024 slots (by wave ballots: the lanes of equal
// expert are the AND of the ballots of its bits) plus the counts of the chunks
// before.  Only whole-number counts are added by atomics, so the order depends on
// nothing but the ids.  Up to kSortSmall slots one workgroup does it all, chunk
// after chunk, in one launch; more take three: counts per chunk, prefix sums over
// the chunks (a wave per expert), places.  32 slots: 3.4 us; 65536 of 128 experts:
// 9.7 us (the gather behind it: 139).
constexpr int kChunk = 1024;
constexpr int kChunkWaves = kChunk / 64;
constexpr int kMaxBuckets = GQ_MAX_EXPERTS + 1;
constexpr int64_t kSortSmall = 4 * kChunk;

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

// Rank of this thread's slot (if in) among those of bucket b in the workgroup's
// chunk.  cnt: (E + 1) * waves counts in LDS; tot[bucket]: the chunk's counts.
__device__ inline int rank_in_chunk(int b, bool in, int E, int bits, unsigned short *cnt, int *tot)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nb = E + 1, nt = blockDim.x, nw = nt >> 6;
    for (int i = threadIdx.x; i < nb * nw; i += nt) cnt[i] = 0;
    __syncthreads();
    const unsigned long long same = same_bucket(b, bits, __ballot(in));
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (in && rank == 0) cnt[wave * nb + b] = (unsigned short)__popcll(same);
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += nt) {
        int s = 0;
        for (int w = 0; w < nw; ++w) {
            const int c = cnt[w * nb + i];
            cnt[w * nb + i] = (unsigned short)s;
            s += c;
        }
        tot[i] = s;
    }
    __syncthreads();
    return in ? rank + cnt[wave * nb + b] : 0;
}

__device__ inline int wave_inclusive(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// base[i] = v[0] + .. + v[i - 1] for i < n, by the first wave; v may be base.
// Ends with the workgroup synchronised.
__device__ inline void exclusive_scan(int *base, const int *v, int n)
{
    if (threadIdx.x < 64) {
        int carry = 0;
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int i = i0 + (int)threadIdx.x;
            const int c = i < n ? v[i] : 0;
            const int inc = wave_inclusive(c);
            if (i < n) base[i] = carry + inc - c;
            carry += __shfl(inc, 63);
        }
    }
    __syncthreads();
}

template <typename TI>
__global__ __launch_bounds__(kChunk) void sort_small_kernel(int *offsets, int *order, int *pos, const TI *ids, int n,
                                                            int E, int bits)
{
    extern __shared__ unsigned short cnt[];
    __shared__ int base[kMaxBuckets], tot[kMaxBuckets];
    const int nb = E + 1, nt = blockDim.x;
    for (int b = threadIdx.x; b < nb; b += nt) tot[b] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += nt) atomicAdd(&tot[bucket_of(ids, i, E)], 1);
    __syncthreads();
    exclusive_scan(base, tot, nb);
    for (int b = threadIdx.x; b < nb; b += nt) offsets[b] = base[b];
    for (int i0 = 0; i0 < n; i0 += nt) {
        const int i = i0 + (int)threadIdx.x;
        const bool in = i < n;
        const int b = in ? bucket_of(ids, i, E) : E;
        const int rank = rank_in_chunk(b, in, E, bits, cnt, tot);
        if (in) {
            const int p = base[b] + rank;
            order[p] = b < E ? i : -1;
            pos[i] = b < E ? p : -1;
        }
        __syncthreads();
        for (int j = threadIdx.x; j < nb; j += nt) base[j] += tot[j];
        // the next chunk's first barrier orders this before its reads
    }
}

// hist[chunk][bucket] = the chunk's slots of each bucket.
template <typename TI>
__global__ __launch_bounds__(kChunk) void sort_count_kernel(int *hist, const TI *ids, int64_t n, int E)
{
    __shared__ int tot[kMaxBuckets];
    for (int b = threadIdx.x; b <= E; b += kChunk) tot[b] = 0;
    __syncthreads();
    const int64_t i = (int64_t)blockIdx.x * kChunk + threadIdx.x;
    if (i < n) atomicAdd(&tot[bucket_of(ids, i, E)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b <= E; b += kChunk) hist[(int64_t)blockIdx.x * (E + 1) + b] = tot[b];
}

// One wave per bucket: its counts become the number in the chunks before, its
// total goes behind the last chunk (hist[chunks][bucket]).
__global__ __launch_bounds__(64) void sort_prefix_kernel(int *hist, int chunks, int E)
{
    const int b = blockIdx.x, nb = E + 1;
    int carry = 0;
    for (int w0 = 0; w0 < chunks; w0 += 64) {
        const int w = w0 + (int)threadIdx.x;
        const int c = w < chunks ? hist[(int64_t)w * nb + b] : 0;
        const int inc = wave_inclusive(c);
        if (w < chunks) hist[(int64_t)w * nb + b] = carry + inc - c;
        carry += __shfl(inc, 63);
    }
    if (threadIdx.x == 0) hist[(int64_t)chunks * nb + b] = carry;
}

template <typename TI>
__global__ __launch_bounds__(kChunk) void sort_place_kernel(int *offsets, int *order, int *pos, const int *hist,
                                                            const TI *ids, int64_t n, int E, int bits)
{
    extern __shared__ unsigned short cnt[];
    __shared__ int base[kMaxBuckets], tot[kMaxBuckets];
    const int nb = E + 1;
    exclusive_scan(base, hist + (int64_t)gridDim.x * nb, nb);
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < nb; b += kChunk) offsets[b] = base[b];
    const int64_t i = (int64_t)blockIdx.x * kChunk + threadIdx.x;
    const bool in = i < n;
    const int b = in ? bucket_of(ids, i, E) : E;
    const int rank = rank_in_chunk(b, in, E, bits, cnt, tot);
    if (!in) return;
    const int p = base[b] + hist[(int64_t)blockIdx.x * nb + b] + rank;
    order[p] = b < E ? (int)i : -1;
    pos[i] = b < E ? p : -1;
}

template <typename TI>
hipError_t launch_sort(int *offsets, int *order, int *pos, const TI *ids, int64_t n, int E, int *hist, hipStream_t s)
{
    const int chunks = (int)((n + kChunk - 1) / kChunk);
    int bits = 0;
    while ((1 << bits) < E + 1) ++bits;
    if (n <= kSortSmall) {
        const int nt = n >= kChunk ? kChunk : n > 64 ? (int)((n + 63) / 64) * 64 : 64;
        hipLaunchKernelGGL(sort_small_kernel<TI>, dim3(1), dim3(nt), sizeof(unsigned short) * (nt / 64) * (E + 1), s,
                           offsets, order, pos, ids, (int)n, E, bits);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(sort_count_kernel<TI>, dim3(chunks), dim3(kChunk), 0, s, hist, ids, n, E);
    hipLaunchKernelGGL(sort_prefix_kernel, dim3(E + 1), dim3(64), 0, s, hist, chunks, E);
    hipLaunchKernelGGL(sort_place_kernel<TI>, dim3(chunks), dim3(kChunk),
                       sizeof(unsigned short) * kChunkWaves * (E + 1), s, offsets, order, pos, hist, ids, n, E, bits);
    return hipGetLastError();
}

// ---------------------------------------------------------------- rows
// A thread takes V consecutive columns of a row: 16 bytes, whatever the row's
// alignment (memory takes unaligned accesses), or one element where a row is
// shorter than that.  The last thread of a row moves back to end with it, and
// repeats what its neighbour does.  A token's rows are taken KR at a time with
// all their loads in flight: a slot without a row reads zeros from a line of its
// own rather than branch, since a branch between loads makes the compiler wait
// for those before it (8192 x 8 rows of 5120 bf16 combined with such branches:
// 210 us).
constexpr int kMaxRowThreads = 512;
__device__ __attribute__((aligned(16))) const unsigned kZeros[4] = {0, 0, 0, 0};

template <typename T, int V> struct Vec {
    T v[V];
};
template <typename T, int V> __device__ inline Vec<T, V> load_vec(const T *p)
{
    Vec<T, V> r;
    __builtin_memcpy(&r, p, sizeof r);
    return r;
}
template <typename T, int V> __device__ inline void store_vec(T *p, const Vec<T, V> &r) { __builtin_memcpy(p, &r, sizeof r); }

// Row of slot t k + j, or -1 (past k, dropped, or outside the rows).
__device__ inline int64_t row_of(const int *pos, int64_t t, int j, int k, int64_t rows)
{
    const int p = pos[t * k + min(j, k - 1)];
    return j < k && p >= 0 && p < rows ? p : -1;
}
template <typename T, int V> __device__ inline Vec<T, V> load_row(const T *Y, int64_t ldy, int64_t p, int64_t c)
{
    return load_vec<T, V>(p >= 0 ? Y + p * ldy + c : (const T *)kZeros);
}

// Each token's row read once and written to its places.
template <typename T, int V, int KR>
__global__ __launch_bounds__(kMaxRowThreads) void gather_kernel(T *Xs, int64_t lds, const T *X, int64_t ldx,
                                                                const int *pos, int64_t rows, int64_t Tn, int k, int64_t D)
{
    const int64_t t = grid_row(), c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V, c = min(c0, D - V);
    if (t >= Tn || c0 >= D) return;
    const Vec<T, V> x = load_vec<T, V>(X + t * ldx + c);
    for (int j0 = 0; j0 < k; j0 += KR) {
        int64_t p[KR];
#pragma unroll
        for (int j = 0; j < KR; ++j) p[j] = row_of(pos, t, j0 + j, k, rows);
#pragma unroll
        for (int j = 0; j < KR; ++j)
            if (p[j] >= 0) store_vec(Xs + p[j] * lds + c, x);
    }
}

template <typename T, int V, int KR>
__global__ __launch_bounds__(kMaxRowThreads) void combine_kernel(T *out, int64_t ldo, const T *Y, int64_t ldy,
                                                                 const int *pos, const float *w, int64_t rows,
                                                                 int64_t Tn, int k, int64_t D)
{
    const int64_t t = grid_row(), c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V, c = min(c0, D - V);
    if (t >= Tn || c0 >= D) return;
    float acc[V] = {};
    for (int j0 = 0; j0 < k; j0 += KR) {
        Vec<T, V> y[KR];
        float wt[KR];
#pragma unroll
        for (int j = 0; j < KR; ++j) {
            const int64_t p = row_of(pos, t, j0 + j, k, rows);
            wt[j] = p < 0 ? 0.0f : w ? w[t * k + j0 + j] : 1.0f;
            y[j] = load_row<T, V>(Y, ldy, p, c);
        }
#pragma unroll
        for (int j = 0; j < KR; ++j)
#pragma unroll
            for (int u = 0; u < V; ++u) acc[u] = fmaf(wt[j], (float)y[j].v[u], acc[u]);
    }
    Vec<T, V> o;
#pragma unroll
    for (int u = 0; u < V; ++u) o.v[u] = (T)acc[u];
    store_vec(out + t * ldo + c, o);
}

// One token per workgroup: dY = w dout for each of its rows, and the dot products
// of dout with them, added over the workgroup in wave order.
template <typename T, int V, int KR>
__global__ __launch_bounds__(kMaxRowThreads) void combine_backward_kernel(T *dY, int64_t lddy, float *dw, const T *dout,
                                                                          int64_t ldo, const T *Y, int64_t ldy,
                                                                          const int *pos, const float *w, int64_t rows,
                                                                          int64_t Tn, int k, int64_t D)
{
    __shared__ float red[kMaxRowThreads / 64][KR];
    const int64_t t = grid_row();
    if (t >= Tn) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
    for (int j0 = 0; j0 < k; j0 += KR) {
        int64_t p[KR];
        float wt[KR], dot[KR] = {};
#pragma unroll
        for (int j = 0; j < KR; ++j) {
            p[j] = row_of(pos, t, j0 + j, k, rows);
            wt[j] = w[t * k + min(j0 + j, k - 1)];
        }
        for (int64_t c0 = threadIdx.x * V; c0 < D; c0 += blockDim.x * V) {
            const int64_t c = min(c0, D - V);
            Vec<T, V> g = load_vec<T, V>(dout + t * ldo + c), y[KR];
#pragma unroll
            for (int j = 0; j < KR; ++j) y[j] = load_row<T, V>(Y, ldy, p[j], c);
#pragma unroll
            for (int j = 0; j < KR; ++j) {
                Vec<T, V> o;
#pragma unroll
                for (int u = 0; u < V; ++u) {
                    // columns its neighbour has added are not added again
                    dot[j] = fmaf(c + u >= c0 ? (float)g.v[u] : 0.0f, c + u >= c0 ? (float)y[j].v[u] : 0.0f, dot[j]);
                    o.v[u] = (T)(wt[j] * (float)g.v[u]);
                }
                if (p[j] >= 0) store_vec(dY + p[j] * lddy + c, o);
            }
        }
#pragma unroll
        for (int j = 0; j < KR; ++j) {
            float d = dot[j];
#pragma unroll
            for (int x = 32; x; x >>= 1) d += __shfl_xor(d, x);
            if (lane == 0) red[wave][j] = d;
        }
        __syncthreads();
        if (threadIdx.x < KR && j0 + (int)threadIdx.x < k) {
            float s = red[0][threadIdx.x];
            for (int i = 1; i < nw; ++i) s += red[i][threadIdx.x];
            dw[t * k + j0 + threadIdx.x] = row_of(pos, t, j0 + threadIdx.x, k, rows) >= 0 ? s : 0.0f;
        }
        __syncthreads();
    }
}

// Threads for a row of D elements, V each: equal passes of at most kMaxRowThreads.
int row_threads(int64_t D, int V, int64_t *passes)
{
    const int64_t nv = (D + V - 1) / V;
    const int64_t np = (nv + kMaxRowThreads - 1) / kMaxRowThreads;
    const int nt = (int)(((nv + np - 1) / np + 63) / 64) * 64;
    *passes = (nv + nt - 1) / nt;
    return nt;
}

// Calls f<V, KR>: V for rows of D elements, KR for k choices.
template <typename T, typename F> hipError_t by_shape(int64_t D, int k, F f)
{
    constexpr int V = 16 / sizeof(T);
    if (D < V) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
    if (k <= 2) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 2>{});
    if (k <= 4) return f(std::integral_constant<int, V>{}, std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, V>{}, std::integral_constant<int, 8>{});
}

template <typename T>
hipError_t launch_gather(T *Xs, int64_t lds, const T *X, int64_t ldx, const int *pos, int64_t rows, int64_t Tn, int k,
                         int64_t D, hipStream_t s)
{
    return by_shape<T>(D, k, [&](auto V, auto KR) {
        int64_t passes;
        const int nt = row_threads(D, V, &passes);
        hipLaunchKernelGGL((gather_kernel<T, decltype(V)::value, decltype(KR)::value>), tile_grid(passes, Tn), dim3(nt), 0,
                           s, Xs, lds, X, ldx, pos, rows, Tn, k, D);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t launch_combine(T *out, int64_t ldo, const T *Y, int64_t ldy, const int *pos, const float *w, int64_t rows,
                          int64_t Tn, int k, int64_t D, hipStream_t s)
{
    return by_shape<T>(D, k, [&](auto V, auto KR) {
        int64_t passes;
        const int nt = row_threads(D, V, &passes);
        hipLaunchKernelGGL((combine_kernel<T, decltype(V)::value, decltype(KR)::value>), tile_grid(passes, Tn), dim3(nt), 0,
                           s, out, ldo, Y, ldy, pos, w, rows, Tn, k, D);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t launch_combine_backward(T *dY, int64_t lddy, float *dw, const T *dout, int64_t ldo, const T *Y, int64_t ldy,
                                   const int *pos, const float *w, int64_t rows, int64_t Tn, int k, int64_t D,
                                   hipStream_t s)
{
    return by_shape<T>(D, k, [&](auto V, auto KR) {
        int64_t passes;
        const int nt = row_threads(D, V, &passes);
        hipLaunchKernelGGL((combine_backward_kernel<T, decltype(V)::value, decltype(KR)::value>), tile_grid(1, Tn), dim3(nt),
                           0, s, dY, lddy, dw, dout, ldo, Y, ldy, pos, w, rows, Tn, k, D);
        return hipGetLastError();
    });
}

int done(hipError_t e)
{
    return e == hipSuccess ? set_error(GQ_OK, "") : set_error(GQ_ERR_HIP, hipGetErrorString(e));
}

// Sizes every call of this file shares; rows is the number of rows of the sorted matrix.
int check_rows(int dtype, int64_t T, int64_t k, int64_t rows, int64_t D)
{
    if (dtype != GQ_F32 && dtype != GQ_BF16) return set_error(GQ_ERR_INVALID_ARG, "unknown dtype");
    if (T < 0 || k < 1 || rows < 0 || D < 1 || D > (1 << 30)) return set_error(GQ_ERR_INVALID_ARG, "bad sizes");
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
    return n <= kSortSmall ? 0 : (size_t)((n + kChunk - 1) / kChunk + 1) * (size_t)(E + 1) * sizeof(int);
}

int experts_sort(int32_t *offsets, int32_t *order, int32_t *pos, const void *ids, int id_bytes, int64_t n, int64_t E,
                 void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (id_bytes != 4 && id_bytes != 8) return set_error(GQ_ERR_INVALID_ARG, "ids must be of 4 or 8 bytes");
    if (n < 0 || n > INT32_MAX) return set_error(GQ_ERR_INVALID_ARG, "bad number of slots");
    if (E < 1 || E > GQ_MAX_EXPERTS) return set_error(GQ_ERR_INVALID_ARG, "E must be 1 .. GQ_MAX_EXPERTS");
    if (!offsets || (n && (!order || !pos || !ids))) return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    const size_t need = experts_sort_workspace_size(n, E);
    if (need && !ws) return set_error(GQ_ERR_INVALID_ARG, "null workspace");
    if (ws_bytes < need) return set_error(GQ_ERR_INVALID_ARG, "workspace too small");
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
