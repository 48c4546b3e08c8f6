// int4_skinny.hip -- int4 / NF4 pack products of few rows: a decoding step, where
// the pack's bytes are the work.
//
// A workgroup takes 16 MT rows by 16 NT columns of Y; its waves share the K range
// in units of 128 k, each with its own loads some units ahead, and add their
// sums through LDS in wave order.  X comes straight from memory (a few rows, in
// L2), the codes too: each byte is read once per 16 MT rows.  The matrix
// instruction runs with up to 15 idle rows, which cost nothing here.
#include "int4mm.h"

namespace gq {
namespace {

constexpr int KU = 128, NH = KU / 32;

template <typename TX, int WMODE, int NG, int MT, int NT, int W, int D>
__global__ __launch_bounds__(64 * W) void int4_skinny_kernel(I4Args a)
{
    constexpr int PX = XParts<TX>::n, PW = WParts<WMODE>::n, XV = 8 * (int)sizeof(TX) / 16;
    __shared__ float red[W][MT * NT * 256];
    __shared__ Nf4Table tab;
    if constexpr (WMODE != W_INT4) {
        tab.fill();
        __syncthreads();
    }
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, 16 * MT, grid_row(), rt)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4, K = a.K;
    const int n0 = blockIdx.x * 16 * NT;
    const int ngroups = K / a.G, lg = __builtin_ctz(a.G);
    const TX *x[MT];
    const uint8_t *c[NT];
    const float *sc[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = (const TX *)a.X + min(rt.r0 + 16 * i + r, rt.r1 - 1) * a.ldx;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = rt.e * a.N + min(n0 + 16 * j + r, a.N - 1);
        c[j] = a.codes + n * (K / 2);
        sc[j] = a.scales + n * ngroups;
    }
    struct Unit {
        u32x4 x[MT][NH][XV];
        unsigned c[NT][NH];
        float s[NT][NG];
    } buf[D];
    // this lane's first k of step h (which 8 k a lane feeds is free as long as X
    // and W agree): one load of codes where the unit is one group
    auto k_of = [&](int h) { return NG == 1 ? 32 * q + 8 * h : 32 * h + 8 * q; };
    auto load = [&](int u, Unit &b) {
        const int k0 = u * KU;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if constexpr (NG == 1) {
                __builtin_memcpy(&b.c[j][0], c[j] + k0 / 2 + 16 * q, 16);
            } else {
#pragma unroll
                for (int h = 0; h < NH; ++h) __builtin_memcpy(&b.c[j][h], c[j] + min(k0 / 2 + 16 * h + 4 * q, K / 2 - 4), 4);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) b.s[j][g] = sc[j][min((k0 + g * (KU / NG)) >> lg, ngroups - 1)];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const int k = k0 + k_of(h);
                if (NG == 1 || k < K) __builtin_memcpy(&b.x[i][h], x[i] + k, 8 * sizeof(TX));
                else
#pragma unroll
                    for (int v = 0; v < XV; ++v) b.x[i][h][v] = u32x4{};
            }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{};
    auto multiply = [&](const Unit &b) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f32x4 part[MT][NT] = {};
#pragma unroll
            for (int h = g * (NH / NG); h < (g + 1) * (NH / NG); ++h) {
                bf16x8 wp[NT][PW];
#pragma unroll
                for (int j = 0; j < NT; ++j) code_parts<WMODE>(b.c[j][h], tab, wp[j]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    bf16x8 xp[PX];
                    if constexpr (PX == 1) xp[0] = __builtin_bit_cast(bf16x8, b.x[i][h][0]);
                    else x_parts(__builtin_bit_cast(f32x4, b.x[i][h][0]), __builtin_bit_cast(f32x4, b.x[i][h][XV - 1]), xp);
#pragma unroll
                    for (int j = 0; j < NT; ++j) part[i][j] = mma_parts(xp, wp[j], part[i][j]);
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        acc[i][j][t] = fmaf(b.s[j][g] * (1.0f / CodeScale<WMODE>::v), part[i][j][t], acc[i][j][t]);
        }
    };
    const int units = (K + KU - 1) / KU;
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (wave + W * d < units) load(wave + W * d, buf[d]);
    for (int u = wave; u < units; u += W * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (u + W * d < units) multiply(buf[d]);
            if (u + W * (d + D) < units) load(u + W * (d + D), buf[d]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) red[wave][(i * 16 + 4 * q + t) * 16 * NT + 16 * j + r] = acc[i][j][t];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * NT * 256; e += 64 * W) {
        float v = red[0][e];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[w][e];
        const int64_t row = rt.r0 + e / (16 * NT);
        const int n = n0 + e % (16 * NT);
        if (row < rt.r1 && n < a.N) store_row(a, row, n, v);
    }
}

template <typename TX, int WMODE, int NG> hipError_t by_rows(const I4Args &a, hipStream_t s)
{
    const bool ex = a.offsets != nullptr;
    auto go = [&](auto kernel, int mt, int nt, int waves) {
        hipLaunchKernelGGL(kernel, tile_grid((a.N + 16 * nt - 1) / (16 * nt), row_tiles(ex, a.E, a.M, 16 * mt)), dim3(64 * waves), 0, s, a);
        return hipGetLastError();
    };
    const int64_t rows = ex ? (a.M + a.E - 1) / a.E : a.M;
    if (rows <= 16) return go(int4_skinny_kernel<TX, WMODE, NG, 1, 1, 8, 2>, 1, 1, 8);
    if (rows <= 32) return go(int4_skinny_kernel<TX, WMODE, NG, 2, 1, 8, 2>, 2, 1, 8);
    return go(int4_skinny_kernel<TX, WMODE, NG, 4, 2, 4, 1>, 4, 2, 4);
}

template <typename TX, int WMODE> hipError_t by_group(const I4Args &a, hipStream_t s)
{
    if (a.G == 128) return by_rows<TX, WMODE, 1>(a, s);
    if (a.G == 64) return by_rows<TX, WMODE, 2>(a, s);
    return by_rows<TX, WMODE, 4>(a, s);
}

}  // namespace

hipError_t launch_int4_skinny(const I4Args &a, bool x_bf16, bool nf4, hipStream_t s)
{
    if (!x_bf16) return nf4 ? by_group<float, W_NF4_3>(a, s) : by_group<float, W_INT4>(a, s);
    if (!nf4) return by_group<__bf16, W_INT4>(a, s);
    return a.y_bf16 ? by_group<__bf16, W_NF4_2>(a, s) : by_group<__bf16, W_NF4_3>(a, s);
}

}  // namespace gq
