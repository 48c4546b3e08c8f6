// int4_tile.hip -- int4 / NF4 pack products of many rows.
//
// Four waves side by side, each PM x PN blocks of 16 x 16 of Y: TM = 16 PM rows by
// TN = 64 PN columns per workgroup, two workgroups to a CU.  A stage is 256 bytes
// of each row of X (128 k of bf16, 64 of fp32), two stages in LDS, the next
// copied past the registers while one is multiplied.  Every wave reads the whole
// X tile and turns only its own columns' codes into bf16, in registers: the codes
// never go through LDS, and a code is converted once per TM rows.
//
// v_mfma_f32_16x16x32_bf16 takes 8 k from each lane: step h of a stage k = 32 h +
// 8 (l / 16) .. + 7, within one group, the group's sum formed apart and multiplied
// by its scale.  A lane loads its row's codes 16 bytes at a time and the groups of
// lanes exchange them (transpose4).  Row rho of a stage is 16 chunks of 16 bytes,
// chunk c at position c ^ (rho & 15); a 16-byte LDS read is served 16 lanes at a
// time, rows 0..3 and 12..15 of one group of 16 lanes with rows 4..11 of the next,
// and neighbouring groups' chunks differ in their low two bits only, so the 16
// meet different positions (a lane with 4 consecutive chunks instead: half of the
// LDS's busy cycles were conflicts).
//
// 8192 x 8192 x 8192, groups of 128, bf16: 1.03 ms, 1.07 PFLOP/s, where the bf16
// matrix cores reach 1.22 in a large library product without the codes.  A wave's
// 128 rows amortise a code's two conversion instructions; its sums and converted
// weights take the registers of two waves per SIMD, so conversions of one
// workgroup run beside the matrix instructions of the other.
#include "int4mm.h"

namespace gq {
namespace {

constexpr int kRow = 256;                   // bytes of X per row and stage

template <typename TX, int WMODE, int NG, int PM, int PN>
__global__ __launch_bounds__(256, 2) void int4_tile_kernel(I4Args a, int64_t nt, int64_t mt, bool dma)
{
    constexpr int NW = 4, TM = 16 * PM, TN = 16 * NW * PN, KS = kRow / (int)sizeof(TX), NH = KS / 32;
    constexpr int kSlot = TM * kRow, NC = TM / (4 * NW), PX = XParts<TX>::n, PW = WParts<WMODE>::n;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    __shared__ Nf4Table tab;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if constexpr (WMODE != W_INT4) tab.fill<PW>();
    int64_t ti, tj;
    grouped_tile(blockIdx.x, nt, mt, ti, tj);
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, TM, ti, rt)) return;
    const int n0 = (int)tj * TN, K = a.K;
    const int mrows = (int)(rt.r1 - rt.r0);
    const uint8_t *xbase = (const uint8_t *)((const TX *)a.X + rt.r0 * a.ldx);
    const int r = lane & 15, q = lane >> 4;

    // copy u: rows 4 wave + 16 u .. + 3; lane l takes position l % 16 of row
    // l / 16.  The offsets are formed at each copy: kept, they would not fit the
    // registers beside the sums.  Rows past the end repeat the last.
    int crow = 4 * wave + q;
    const unsigned ch = 16u * (r ^ (crow & 15));
    const unsigned ld = (unsigned)(a.ldx * (int64_t)sizeof(TX));
    const unsigned lbase = lds_offset(lds);
    const int kbytes = K * (int)sizeof(TX);
    auto copy = [&](int b, int slot) {
        asm volatile("" : "+v"(crow));
        if (dma && (b + 1) * kRow <= kbytes) {
#pragma unroll
            for (int u = 0; u < NC; ++u)
                copy16_lds(xbase + kRow * b, (unsigned)min(crow + 16 * u, mrows - 1) * ld + ch,
                           lbase + slot * kSlot + (4 * wave + 16 * u) * kRow);
        } else {
            // rows that do not start on 16 bytes, or the end of a row: through registers, zero past K
#pragma unroll
            for (int u = 0; u < NC; ++u)
                *(u32x4 *)(lds + slot * kSlot + (4 * wave + 16 * u) * kRow + 16 * lane) =
                    load16(xbase + kRow * b + ((unsigned)min(crow + 16 * u, mrows - 1) * ld + ch), kbytes - kRow * b - (int)ch);
        }
    };

    const uint8_t *cbase = a.codes + (rt.e * a.N + n0) * (int64_t)(K / 2);
    const int ngroups = K / a.G, lg = __builtin_ctz(a.G);
    const float *sbase = a.scales + (rt.e * a.N + n0) * (int64_t)ngroups;
    const int nlast = a.N - n0 - 1;
    int nrow = 16 * PN * wave + r;
    unsigned cn[PN][NH];
    float sn[PN][NG];
    auto load_w = [&](int b) {
        asm volatile("" : "+v"(nrow));
        // past K: any codes of the row (X is zero there)
#pragma unroll
        for (int j = 0; j < PN; ++j) {
            const unsigned n = (unsigned)min(nrow + 16 * j, nlast);
            const uint8_t *c = cbase + n * (unsigned)(K / 2);
            if constexpr (NH == 4) {
                __builtin_memcpy(&cn[j][0], c + min((KS / 2) * b + 16 * q, K / 2 - 16), 16);
            } else {
#pragma unroll
                for (int h = 0; h < NH; ++h) __builtin_memcpy(&cn[j][h], c + min((KS / 2) * b + 16 * h + 4 * q, K / 2 - 4), 4);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) sn[j][g] = sbase[n * (unsigned)ngroups + min((b * KS + g * (KS / NG)) >> lg, ngroups - 1)];
        }
    };
    f32x4 acc[PM][PN];
#pragma unroll
    for (int i = 0; i < PM; ++i)
#pragma unroll
        for (int j = 0; j < PN; ++j) acc[i][j] = f32x4{};
    const int nb = (K + KS - 1) / KS;
    copy(0, 0);
    load_w(0);
    for (int b = 0; b < nb; ++b) {
        const int slot = b & 1;
        publish();
        bf16x8 w[PN][NH][PW];
        float s[PN][NG];
#pragma unroll
        for (int j = 0; j < PN; ++j) {
            if constexpr (NH == 4) transpose4(cn[j]);
#pragma unroll
            for (int h = 0; h < NH; ++h) code_parts<WMODE>(cn[j][h], tab, w[j][h]);
#pragma unroll
            for (int g = 0; g < NG; ++g) s[j][g] = sn[j][g] * (1.0f / CodeScale<WMODE>::v);
        }
        if (b + 1 < nb) {
            copy(b + 1, slot ^ 1);
            load_w(b + 1);
        }
        const uint8_t *xs = lds + slot * kSlot + r * kRow;
#pragma unroll
        for (int i = 0; i < PM; ++i) {
            bf16x8 x[NH][PX];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                // element of the row's stage at which this lane's 8 begin, and its chunk
                const int k0 = 32 * h + 8 * q;
                const int c = k0 * (int)sizeof(TX) / 16;
                x_parts((const TX *)(xs + 16 * i * kRow + 16 * (c ^ r)), (const TX *)(xs + 16 * i * kRow + 16 * ((c + 1) ^ r)), x[h]);
            }
#pragma unroll
            for (int j0 = 0; j0 < PN; j0 += 2)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    f32x4 part[2] = {};
#pragma unroll
                    for (int h = g * (NH / NG); h < (g + 1) * (NH / NG); ++h)
#pragma unroll
                        for (int j = 0; j < 2; ++j) part[j] = mma_parts(x[h], w[j0 + j][h], part[j]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[i][j0 + j][t] = fmaf(s[j0 + j][g], part[j][t], acc[i][j0 + j][t]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < PM; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t row = rt.r0 + 16 * i + 4 * q + t;
            if (row >= rt.r1) continue;
#pragma unroll
            for (int j = 0; j < PN; ++j) {
                const int n = n0 + 16 * (PN * wave + j) + r;
                if (n < a.N) store_row(a, row, n, acc[i][j][t]);
            }
        }
}

template <typename TX, int WMODE, int NG, int PM, int PN> hipError_t launch(const I4Args &a, hipStream_t s)
{
    constexpr int TM = 16 * PM, TN = 64 * PN;
    constexpr size_t lds = 2 * (size_t)TM * kRow;
    constexpr auto kernel = int4_tile_kernel<TX, WMODE, NG, PM, PN>;
    const hipError_t e = allow_lds<kernel>(lds);
    if (e != hipSuccess) return e;
    const bool dma = ((uintptr_t)a.X & 15) == 0 && (a.ldx * sizeof(TX)) % 16 == 0;
    const int64_t nt = (a.N + TN - 1) / TN, mt = row_tiles(a.offsets != nullptr, a.E, a.M, TM);
    if (!grid_fits(nt * mt, 256)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(nt * mt)), dim3(256), lds, s, a, nt, mt, dma);
    return hipGetLastError();
}

// Tile shapes by number: 128 x 256, 128 x 128, 96 x 128, 64 x 128.  The weights'
// bf16 parts of a stage stay in registers beside the sums: 256 columns fit with
// one part and up to two scales per stage.
template <typename TX, int WMODE, int NG> hipError_t by_shape(const I4Args &a, int shape, hipStream_t s)
{
    if constexpr (WMODE == W_INT4 && NG <= 2) {
        if (shape == 0) return launch<TX, WMODE, NG, 8, 4>(a, s);
    }
    if (shape <= 1) return launch<TX, WMODE, NG, 8, 2>(a, s);
    if (shape == 2) return launch<TX, WMODE, NG, 6, 2>(a, s);
    return launch<TX, WMODE, NG, 4, 2>(a, s);
}

template <typename TX, int WMODE> hipError_t by_group(const I4Args &a, int shape, hipStream_t s)
{
    constexpr int KS = kRow / (int)sizeof(TX);
    if (a.G >= KS) return by_shape<TX, WMODE, 1>(a, shape, s);
    if (2 * a.G == KS) return by_shape<TX, WMODE, 2>(a, shape, s);
    if constexpr (KS == 128) return by_shape<TX, WMODE, 4>(a, shape, s);
    return hipErrorInvalidValue;
}

}  // namespace

// The larger tile does less work per product, the smaller leaves fewer CUs idle.
// `slots` workgroups of a shape run at a time; a round of up to 256 takes `few`
// us, a full one `full` (bf16 rows, K = 5120, measured at M = 128 .. 8192).
double int4_tile_cost(const I4Args &a, bool x_bf16, bool nf4, int *shape)
{
    static const struct { int tm, tn, slots; double few, full; } kShapes[4] = {
        {128, 256, 512, 133, 160}, {128, 128, 512, 82, 86}, {96, 128, 768, 63, 98}, {64, 128, 1024, 52, 104}};
    const bool wide = !nf4 && a.G >= (x_bf16 ? 64 : 32);
    double best = 0;
    for (int i = wide ? 0 : 1; i < 4; ++i) {
        const auto &k = kShapes[i];
        const int64_t t = (a.N + k.tn - 1) / k.tn * row_tiles(a.offsets != nullptr, a.E, a.M, k.tm);
        const int64_t rem = t % k.slots;
        double c = (double)(t / k.slots) * k.full;
        if (rem) c += rem <= 256 ? k.few : k.few + (k.full - k.few) * (double)(rem - 256) / (double)(k.slots - 256);
        if (best == 0 || c < best) { best = c; *shape = i; }
    }
    return best;
}

hipError_t launch_int4_tile(const I4Args &a, bool x_bf16, bool nf4, int shape, hipStream_t s)
{
    if (!x_bf16) return nf4 ? by_group<float, W_NF4_3>(a, shape, s) : by_group<float, W_INT4>(a, shape, s);
    if (!nf4) return by_group<__bf16, W_INT4>(a, shape, s);
    return a.y_bf16 ? by_group<__bf16, W_NF4_2>(a, shape, s) : by_group<__bf16, W_NF4_3>(a, shape, s);
}

}  // namespace gq
