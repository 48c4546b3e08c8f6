// int4_skinny.hip -- int4 / NF4 pack products of 3 to 64 rows, where the pack's
// bytes are still most of the work but fp32 dot products no longer keep up.
//
// A workgroup takes 16 MT rows by 16 NT columns of Y; its waves take a range of K
// each, in units of 128 k, and add their sums through LDS in wave order.  Each
// code is read once per 16 MT rows, X once per 16 NT columns (from L2), and what
// bounds the kernel is how many cache lines its loads touch: a matrix operand
// loaded as it is used takes 16 rows by 64 bytes, 16 half lines, so X goes
// through LDS in whole lines instead (16 x 5120 x 10240: 20.7 -> 13.4 us).  Codes
// and scales take the same way, so that the waits are the ring's own: the
// compiler's, which does not know of the copies, would wait for those too.  The
// ring is the wave's own part of LDS, with no barrier; a deeper one leaves fewer
// workgroups to a CU (16 x 10240 x 5120: 13.4 / 14.0 / 17.7 us with 2, 3, 4 slots).
#include "int4mm.h"

namespace gq {
namespace {

constexpr int KU = 128, NH = KU / 32;

// XC: copies of X per unit, 1 KiB each; rows past them (there are none) hold
// whatever was in LDS, in rows of Y that are not stored.
template <typename TX, int WMODE, int NG, int MT, int NT, int W, int XC>
__global__ __launch_bounds__(64 * W) void int4_skinny_kernel(I4Args a)
{
    constexpr int PX = XParts<TX>::n, PW = WParts<WMODE>::n;
    constexpr int ROWB = KU * (int)sizeof(TX), RC = 1024 / ROWB;            // bytes per row, rows per copy
    constexpr int XB = 16 * MT * ROWB, SLOT = XB + NT * (1024 + 256);               // X, codes, scales
    static_assert(XC * RC <= 16 * MT, "copies");
    static_assert(2 * SLOT >= MT * NT * 1024, "the sums reuse the ring's space");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    __shared__ Nf4Table tab;
    if constexpr (WMODE != W_INT4) {
        tab.fill<PW>();
        __syncthreads();
    }
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, 16 * MT, grid_row(), rt)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4, K = a.K;
    const int n0 = blockIdx.x * 16 * NT;
    const int ngroups = K / a.G, lg = __builtin_ctz(a.G);
    const int mrows = (int)(rt.r1 - rt.r0);
    const uint8_t *xbase = (const uint8_t *)((const TX *)a.X + rt.r0 * a.ldx);
    const unsigned ld = (unsigned)(a.ldx * (int64_t)sizeof(TX)), kbytes = (unsigned)K * (unsigned)sizeof(TX);
    // copy i: rows RC i .. of the unit; the 16-byte chunk c of row rho lies at
    // position c ^ (rho & 15), so 8 lanes that read one chunk of 8 rows meet 8
    // different positions
    uint8_t *xl = lds + wave * 2 * SLOT;
    const unsigned xlo = lds_offset(xl);
    unsigned xo[XC], xc[XC];
#pragma unroll
    for (int i = 0; i < XC; ++i) {
        const int row = RC * i + lane / (ROWB / 16);
        xo[i] = (unsigned)min(row, mrows - 1) * ld;
        xc[i] = 16u * ((unsigned)(lane % (ROWB / 16)) ^ (row & 15));
    }
    // codes: lane l takes bytes 16 (l % 4) .. of row l / 4's 64; scales: lane l
    // group l / 16 of row l % 16 of the unit
    const int64_t row0 = rt.e * a.N + n0;
    const uint8_t *cbase = a.codes + row0 * (K / 2);
    const float *sbase = a.scales + row0 * ngroups;
    const unsigned cc = 16u * (lane & 3), cend = (unsigned)(K / 2 - 16);
    unsigned co[NT], so[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        co[j] = (unsigned)min(16 * j + (lane >> 2), a.N - n0 - 1) * (unsigned)(K / 2);
        so[j] = (unsigned)min(16 * j + r, a.N - n0 - 1) * (unsigned)ngroups;
    }
    constexpr int LOADS = XC + 2 * NT;
    auto issue = [&](int u, int slot) {
        const unsigned at = xlo + slot * SLOT;
        // K % 128 left over (NG > 1): what lies past the row's end repeats it, to be zeroed
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            const unsigned k = (unsigned)u * ROWB + xc[i];
            copy16_lds(xbase, xo[i] + (NG == 1 ? k : min(k, kbytes - 16)), at + 1024 * i);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            copy16_lds(cbase, co[j] + min((unsigned)u * (KU / 2) + cc, cend), at + XB + 1024 * j);
            copy4_lds(sbase, 4u * (so[j] + (NG == 1 ? u : min(((u * KU) >> lg) + q, ngroups - 1))), at + XB + NT * 1024 + 256 * j);
        }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{};
    // step h of a unit covers k = 32 h + 8 q .. + 7, within one group: the lane's 16
    // bytes of codes, transposed
    auto multiply = [&](int u, int slot) {
        const uint8_t *us = xl + slot * SLOT, *xs = us + r * ROWB;
        unsigned c[NT][NH];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const u32x4 v = *(const u32x4 *)(us + XB + 1024 * j + 64 * r + 16 * q);
#pragma unroll
            for (int h = 0; h < NH; ++h) c[j][h] = v[h];
            transpose4(c[j]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f32x4 part[MT][NT] = {};
#pragma unroll
            for (int h = g * (NH / NG); h < (g + 1) * (NH / NG); ++h) {
                bf16x8 wp[NT][PW];
#pragma unroll
                for (int j = 0; j < NT; ++j) code_parts<WMODE>(c[j][h], tab, wp[j]);
                const bool in = NG == 1 || u * KU + 32 * h < K;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    bf16x8 xp[PX];
                    const int ch = (32 * h + 8 * q) * (int)sizeof(TX) / 16;
                    x_parts((const TX *)(xs + 16 * i * ROWB + 16 * (ch ^ r)), (const TX *)(xs + 16 * i * ROWB + 16 * ((ch + 1) ^ r)), xp);
                    if (NG > 1) {
#pragma unroll
                        for (int p = 0; p < PX; ++p) xp[p] = in ? xp[p] : bf16x8{};
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) part[i][j] = mma_parts(xp, wp[j], part[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float s = *(const float *)(us + XB + NT * 1024 + 256 * j + 4 * (r + 16 * g)) * (1.0f / CodeScale<WMODE>::v);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(s, part[i][j][t], acc[i][j][t]);
            }
        }
    };
    const int units = (K + KU - 1) / KU, per = (units + W - 1) / W;
    const int u0 = wave * per, u1 = min(u0 + per, units);
    ring<LOADS>(u0, u1, issue, multiply);
    __syncthreads();                                     // every wave is past its X
    float *red = (float *)lds;                           // [W][MT * NT * 256]
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) red[wave * MT * NT * 256 + (i * 16 + 4 * q + t) * 16 * NT + 16 * j + r] = acc[i][j][t];
    __syncthreads();
    for (int e = threadIdx.x; e < MT * NT * 256; e += 64 * W) {
        float v = red[e];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[w * MT * NT * 256 + e];
        const int64_t row = rt.r0 + e / (16 * NT);
        const int n = n0 + e % (16 * NT);
        if (row < rt.r1 && n < a.N) store_row(a, row, n, v);
    }
}

template <typename TX, int WMODE, int NG, int MT, int NT, int W, int XC> hipError_t launch(const I4Args &a, hipStream_t s)
{
    constexpr size_t lds = (size_t)W * 2 * (16 * MT * KU * sizeof(TX) + NT * (1024 + 256));
    static_assert(lds + sizeof(Nf4Table) <= 160 * 1024, "LDS");
    constexpr auto kernel = int4_skinny_kernel<TX, WMODE, NG, MT, NT, W, XC>;
    const hipError_t e = allow_lds<kernel>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, tile_grid((a.N + 16 * NT - 1) / (16 * NT), row_tiles(a.offsets != nullptr, a.E, a.M, 16 * MT)),
                       dim3(64 * W), lds, s, a);
    return hipGetLastError();
}

// Tiles of 16 x 16, 16 x 32 and 32 x 32: the larger reads less, the smaller leaves
// fewer CUs idle at the end.
template <typename TX, int WMODE, int NG> hipError_t by_rows(const I4Args &a, int shape, hipStream_t s)
{
    constexpr int C16 = 16 * KU * (int)sizeof(TX) / 1024;        // copies for 16 rows
    if (shape == 2) return launch<TX, WMODE, NG, 2, 2, 4, 2 * C16>(a, s);
    if (a.M <= 4) return shape ? launch<TX, WMODE, NG, 1, 2, 4, C16 / 4>(a, s) : launch<TX, WMODE, NG, 1, 1, 4, C16 / 4>(a, s);
    return shape ? launch<TX, WMODE, NG, 1, 2, 4, C16>(a, s) : launch<TX, WMODE, NG, 1, 1, 4, C16>(a, s);
}

template <typename TX, int WMODE> hipError_t by_group(const I4Args &a, int shape, hipStream_t s)
{
    if (a.G == 128) return by_rows<TX, WMODE, 1>(a, shape, s);
    if (a.G == 64) return by_rows<TX, WMODE, 2>(a, shape, s);
    return by_rows<TX, WMODE, 4>(a, shape, s);
}

}  // namespace

// One tile per CU at a time; a round of tiles of 16 x 16, 16 x 32 or 32 x 32 takes
// 4, 6 or 8 us.
double int4_skinny_cost(const I4Args &a, int *shape)
{
    double best = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t tm = i == 2 ? 32 : 16, tn = i ? 32 : 16;
        const int64_t tiles = (a.N + tn - 1) / tn * row_tiles(a.offsets != nullptr, a.E, a.M, tm);
        const double c = (double)((tiles + 255) / 256 * (4 + 2 * i));
        if (i == 0 || c < best) { best = c; *shape = i; }
    }
    return best;
}

hipError_t launch_int4_skinny(const I4Args &a, bool x_bf16, bool nf4, int shape, hipStream_t s)
{
    if (!x_bf16) return nf4 ? by_group<float, W_NF4_3>(a, shape, s) : by_group<float, W_INT4>(a, shape, s);
    if (!nf4) return by_group<__bf16, W_INT4>(a, shape, s);
    return a.y_bf16 ? by_group<__bf16, W_NF4_2>(a, shape, s) : by_group<__bf16, W_NF4_3>(a, shape, s);
}

}  // namespace gq
