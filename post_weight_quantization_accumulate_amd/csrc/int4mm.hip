// int4mm.hip -- products with the int4 and NF4 packs the quantisers write:
//     Y[m][n] = sum_g s[n][g] sum_{k in group g} X[m][k] v(c[n][k]),
// v(c) the code itself (int4) or its NF4 level.
//
// On the bf16 matrix cores every product has to be of two bf16 numbers: a code is
// one exactly, a bf16 x too; fp32 x and NF4 levels are split into three bf16
// parts of 8 bits, whose products are exact and summed in fp32.  Groups of 32 and
// more are summed apart and scaled once (int4_tile.hip for many rows,
// int4_skinny.hip for few); smaller groups are the kernel of this file.
#include "gq.h"

#include "gemv.h"
#include "int4mm.h"

namespace gq {
namespace {

constexpr int kWaves = 4;

// Elements k .. k + 7 of a row of X as bf16 parts, zero past K.  K8: K % 8 == 0.
template <bool K8, typename TX> __device__ inline void load_x8(const TX *row, int k, int K, bf16x8 (&p)[XParts<TX>::n])
{
    __attribute__((aligned(16))) TX v[8] = {};
    if constexpr (K8) {
        if (k < K) __builtin_memcpy(v, row + k, sizeof v);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (k + t < K) v[t] = row[k + t];
    }
    x_parts(v, v + 4, p);
}

// Codes k .. k + 7 of a row, code t in bits 4t .. 4t + 3, zero past K.
template <bool K8> __device__ inline unsigned load_c8(const uint8_t *row, int k, int K)
{
    unsigned w = 0;
    if constexpr (K8) {
        if (k < K) __builtin_memcpy(&w, row + k / 2, 4);
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (k + 2 * t < K) w |= (unsigned)row[k / 2 + t] << (8 * t);
    }
    return w;
}

// Groups of 1 .. 16: one matrix instruction spans several groups, so the
// dequantised fp32 weight itself is split into bf16 parts.  One 16 x 16 tile of Y
// per workgroup, its K range dealt to the four waves and their sums added
// through LDS in wave order.
template <typename TX, bool NF4, bool K8> __global__ __launch_bounds__(64 * kWaves) void int4_small_group_kernel(I4Args a)
{
    constexpr int PX = XParts<TX>::n;
    __shared__ float red[kWaves][256];
    __shared__ float lut[16];
    if (threadIdx.x < 16) lut[threadIdx.x] = NF4 ? kNF4[threadIdx.x] : (float)((int)(threadIdx.x ^ 8) - 8);
    __syncthreads();
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, 16, grid_row(), rt)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int n = min(n0 + r, a.N - 1);
    const TX *x = (const TX *)a.X + min(rt.r0 + r, rt.r1 - 1) * a.ldx;
    const uint8_t *c = a.codes + (rt.e * a.N + n) * (int64_t)(a.K / 2);
    const float *sc = a.scales + (rt.e * a.N + n) * (int64_t)(a.K / a.G);
    const int lg = __builtin_ctz(a.G);
    f32x4 acc{};
    for (int k0 = 32 * wave; k0 < a.K; k0 += 32 * kWaves) {
        bf16x8 xp[PX], wp[3];
        load_x8<K8>(x, k0 + 8 * q, a.K, xp);
        const unsigned cw = load_c8<K8>(c, k0 + 8 * q, a.K);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int k = k0 + 8 * q + t;
            const float s = k < a.K ? sc[k >> lg] : 0.0f;
            unsigned short p[3];
            weight_parts(lut[(cw >> (4 * t)) & 15] * s, p);
#pragma unroll
            for (int j = 0; j < 3; ++j) wp[j][t] = __builtin_bit_cast(__bf16, p[j]);
        }
        acc = mma_parts(xp, wp, acc);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][64 * i + lane] = acc[i];
    __syncthreads();
    // element (row 4 (lane / 16) + i, column lane % 16) of the tile
    const int i = threadIdx.x >> 6;
    float v = red[0][64 * i + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[w][64 * i + lane];
    const int64_t row = rt.r0 + 4 * q + i;
    if (row < rt.r1 && n0 + r < a.N) store_row(a, row, n0 + r, v);
}

template <typename TX, bool NF4> hipError_t launch_small_group(const I4Args &a, hipStream_t s)
{
    const dim3 grid = tile_grid((a.N + 15) / 16, row_tiles(a.offsets != nullptr, a.E, a.M, 16));
    if (a.K % 8 == 0) hipLaunchKernelGGL((int4_small_group_kernel<TX, NF4, true>), grid, dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL((int4_small_group_kernel<TX, NF4, false>), grid, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_int4(const I4Args &a, bool x_bf16, bool nf4, hipStream_t s)
{
    if (a.G < 32) {
        if (x_bf16) return nf4 ? launch_small_group<__bf16, true>(a, s) : launch_small_group<__bf16, false>(a, s);
        return nf4 ? launch_small_group<float, true>(a, s) : launch_small_group<float, false>(a, s);
    }
    const int64_t rows = a.offsets ? (a.M + a.E - 1) / a.E : a.M;
    GemvArgs v{};
    v.Y = a.Y; v.X = a.X; v.codes = a.codes; v.scales = a.scales; v.offsets = a.offsets;
    v.M = a.M; v.ldx = a.ldx; v.ldy = a.ldy; v.E = a.E;
    v.N = a.N; v.K = a.K; v.G = a.G;
    v.y_bf16 = a.y_bf16; v.x_bf16 = x_bf16;
    const int kind = nf4 ? GEMV_NF4 : GEMV_INT4;
    if (rows <= kGemvMaxRows && gemv_ok(v, kind, (int)rows)) return launch_gemv(v, kind, (int)rows, s);
    int small = 0, large = 0;
    const double cost = int4_tile_cost(a, x_bf16, nf4, &large);
    const bool aligned = ((uintptr_t)a.X & 15) == 0 && (a.ldx * (x_bf16 ? 2 : 4)) % 16 == 0 && ((uintptr_t)a.codes & 15) == 0;
    if (aligned && int4_skinny_cost(a, &small) < cost) return launch_int4_skinny(a, x_bf16, nf4, small, s);
    return launch_int4_tile(a, x_bf16, nf4, large, s);
}

}  // namespace
}  // namespace gq

using namespace gq;

namespace {

int int4_run(void *Y, int y_dtype, int64_t ldy, const void *X, int x_dtype, int64_t ldx, const uint8_t *codes,
             const float *scales, const int32_t *offsets, int64_t E, int64_t M, int64_t N, int64_t K, int64_t group,
             uint32_t flags, hipStream_t stream)
{
    if (flags & ~(uint32_t)(GQ_STATIC_GROUPS | GQ_NF4 | GQ_ACT_ORDER))
        return set_error(GQ_ERR_INVALID_ARG, "unknown flag bits");
    if ((x_dtype != GQ_F32 && x_dtype != GQ_BF16) || (y_dtype != GQ_F32 && y_dtype != GQ_BF16))
        return set_error(GQ_ERR_INVALID_ARG, "unknown dtype");
    if (M < 0 || N < 1) return set_error(GQ_ERR_INVALID_ARG, "M must be >= 0 and N >= 1");
    if (K < 2 || (K & 1)) return set_error(GQ_ERR_INVALID_ARG, "K must be even and >= 2 (two codes per byte)");
    if (group < 1 || group > 128 || (group & (group - 1)) || K % group)
        return set_error(GQ_ERR_INVALID_ARG, "group must be a power of two <= 128 that divides K");
    if (ldx < K || ldy < N) return set_error(GQ_ERR_INVALID_ARG, "a row stride is below the row's length");
    // the kernels' offsets within a tile (128 rows of X, 256 of codes and scales) have 32 bits
    if (M > INT32_MAX || N > (1 << 24) || K > (1 << 22) || ldx > (1 << 22))
        return set_error(GQ_ERR_INVALID_ARG, "size too large");
    if (M == 0) return set_error(GQ_OK, "");
    if (!Y || !X || !codes || !scales) return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    I4Args a{};
    a.Y = Y; a.X = X; a.codes = codes; a.scales = scales; a.offsets = offsets;
    a.M = M; a.ldx = ldx; a.ldy = ldy; a.E = E;
    a.N = (int)N; a.K = (int)K; a.G = (int)group;
    a.y_bf16 = y_dtype == GQ_BF16;
    const bool nf4 = flags & GQ_NF4;
    const hipError_t e = launch_int4(a, x_dtype == GQ_BF16, nf4, stream);
    return e == hipSuccess ? set_error(GQ_OK, "") : set_error(GQ_ERR_HIP, hipGetErrorString(e));
}

}  // namespace

extern "C" {

int int4_matmul(void *Y, int y_dtype, int64_t ldy, const void *X, int x_dtype, int64_t ldx, const uint8_t *codes,
                const float *scales, int64_t M, int64_t N, int64_t K, int64_t group, uint32_t flags,
                hipStream_t stream)
{
    return int4_run(Y, y_dtype, ldy, X, x_dtype, ldx, codes, scales, nullptr, 1, M, N, K, group, flags, stream);
}

int int4_matmul_experts(void *Y, int y_dtype, int64_t ldy, const void *X, int x_dtype, int64_t ldx,
                        const uint8_t *codes, const float *scales, const int32_t *offsets, int64_t E, int64_t M,
                        int64_t N, int64_t K, int64_t group, uint32_t flags, hipStream_t stream)
{
    if (E < 1 || E > GQ_MAX_EXPERTS) return set_error(GQ_ERR_INVALID_ARG, "E must be 1 .. GQ_MAX_EXPERTS");
    if (!offsets) return set_error(GQ_ERR_INVALID_ARG, "null offsets");
    return int4_run(Y, y_dtype, ldy, X, x_dtype, ldx, codes, scales, offsets, E, M, N, K, group, flags, stream);
}

}  // extern "C"
