// int4_skinny.hip -- int4 / NF4 pack products of 3 to 64 rows, where the pack's
// bytes are still most of the work but fp32 dot products no longer keep up.
//
// A workgroup takes 16 MT rows by 16 NT columns of Y; its waves take a range of K
// each, in units of 128 k, and add their sums through LDS in wave order.  Each
// code is read once per 16 MT rows, X once per 16 NT columns (from L2), and what
// bounds the kernel is how many cache lines its loads touch: a matrix operand
// loaded as it is used takes 16 rows by 64 bytes, 16 half lines, so X goes
// through LDS in whole lines instead (16 x 5120 x 10240: 20.7 -> MEASURE us), into
// a part of the wave's own, with no barrier: the wave waits for its own copies.
// A unit's loads are issued while the one before it is multiplied, in a loop
// without branches: at a branch the compiler waits for every load in flight.
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
    constexpr int ROWB = KU * (int)sizeof(TX), RC = 1024 / ROWB, SLOT = 16 * MT * ROWB;   // bytes per row, rows per copy
    static_assert(XC * RC <= 16 * MT, "copies");
    static_assert(2 * SLOT >= MT * NT * 1024, "the sums reuse X's space");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
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
    const uint8_t *c[NT];
    const float *sc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = rt.e * a.N + min(n0 + 16 * j + r, a.N - 1);
        c[j] = a.codes + n * (K / 2);
        sc[j] = a.scales + n * ngroups;
    }
    // step h of a unit covers k = 32 h + 8 q .. + 7, within one group; the codes are
    // loaded 16 bytes to a lane and transposed, the scales of up to 4 groups by the
    // four groups of lanes
    struct Unit {
        unsigned c[NT][NH];
        float s[NT];
    };
    constexpr int LOADS = XC + 2 * NT;                   // memory instructions of a unit
    auto load = [&](int u, Unit &b) {
        const int k0 = u * KU;
        // K % 128 left over (NG > 1): what lies past the row's end repeats it, to be zeroed
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            const unsigned at = (unsigned)u * ROWB + xc[i];
            copy16_lds(xbase, xo[i] + (NG == 1 ? at : min(at, kbytes - 16)), xlo + (u & 1) * SLOT + 1024 * i);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            __builtin_memcpy(&b.c[j][0], c[j] + min(k0 / 2 + 16 * q, K / 2 - 16), 16);
            b.s[j] = sc[j][NG == 1 ? u : min((k0 >> lg) + q, ngroups - 1)];
        }
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{};
    auto multiply = [&](int u, Unit &b) {
        const uint8_t *xs = xl + (u & 1) * SLOT + r * ROWB;
#pragma unroll
        for (int j = 0; j < NT; ++j) transpose4(b.c[j]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f32x4 part[MT][NT] = {};
#pragma unroll
            for (int h = g * (NH / NG); h < (g + 1) * (NH / NG); ++h) {
                bf16x8 wp[NT][PW];
#pragma unroll
                for (int j = 0; j < NT; ++j) code_parts<WMODE>(b.c[j][h], tab, wp[j]);
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
                const float s = (NG == 1 ? b.s[j] : __shfl(b.s[j], r + 16 * g)) * (1.0f / CodeScale<WMODE>::v);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(s, part[i][j][t], acc[i][j][t]);
            }
        }
    };
    const int units = (K + KU - 1) / KU, per = (units + W - 1) / W;
    const int u0 = wave * per, u1 = min(u0 + per, units);
    if (u0 < u1) {
        Unit cur, nxt;
        load(u0, cur);
        for (int u = u0; u + 1 < u1; ++u) {
            asm volatile("" ::: "memory");               // the other slot's reads are done
            load(u + 1, nxt);
            wait_copies<LOADS>();                        // unit u's are in
            multiply(u, cur);
            cur = nxt;
        }
        wait_copies<0>();
        multiply(u1 - 1, cur);
    }
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
    constexpr size_t lds = (size_t)W * 2 * 16 * MT * KU * sizeof(TX);
    const auto kernel = int4_skinny_kernel<TX, WMODE, NG, MT, NT, W, XC>;
    static const bool lds_ok =
        hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) == hipSuccess;
    if (!lds_ok) return hipErrorInvalidConfiguration;
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
    if (a.M <= 4) return shape ? launch<TX, WMODE, NG, 1, 2, 8, C16 / 4>(a, s) : launch<TX, WMODE, NG, 1, 1, 8, C16 / 4>(a, s);
    return shape ? launch<TX, WMODE, NG, 1, 2, 8, C16>(a, s) : launch<TX, WMODE, NG, 1, 1, 8, C16>(a, s);
}

template <typename TX, int WMODE> hipError_t by_group(const I4Args &a, int shape, hipStream_t s)
{
    if (a.G == 128) return by_rows<TX, WMODE, 1>(a, shape, s);
    if (a.G == 64) return by_rows<TX, WMODE, 2>(a, shape, s);
    return by_rows<TX, WMODE, 4>(a, shape, s);
}

}  // namespace

// Time of the whole grid in units of a 16 x 16 tile's fixed part: one tile per CU
// at a time, tiles of 16 x 16, 16 x 32 and 32 x 32 costing 2, 3 and 4.
int64_t int4_skinny_cost(const I4Args &a, int *shape)
{
    int64_t best = 0;
    for (int i = 0; i < 3; ++i) {
        const int64_t tm = i == 2 ? 32 : 16, tn = i ? 32 : 16;
        const int64_t tiles = (a.N + tn - 1) / tn * row_tiles(a.offsets != nullptr, a.E, a.M, tm);
        const int64_t c = (tiles + 255) / 256 * (2 + i);
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
