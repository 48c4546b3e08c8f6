// int4mm.hip -- products with the int4 and NF4 packs the quantisers write:
//     Y[m][n] = sum_g s[n][g] sum_{k in group g} X[m][k] v(c[n][k]),
// v(c) the code itself (int4) or its NF4 level.
#include "gq.h"
#include "gq_internal.h"
#include "matmul.h"

namespace gq {
namespace {

constexpr int kWaves = 4;

struct I4Args {
    void *Y;
    const void *X;
    const uint8_t *codes;
    const float *scales;
    const int *offsets;
    int64_t M, ldx, ldy, E;
    int N, K, G;
};

// Elements k .. k + 7 of a row of X as bf16 parts (one for bf16, three for
// fp32), zero past K.
template <bool VEC> __device__ inline void load_x8(const __bf16 *row, int k, int K, bf16x8 (&p)[1])
{
    if constexpr (VEC) {
        if (k < K) p[0] = *(const bf16x8 *)(row + k);
        else p[0] = bf16x8{};
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) p[0][t] = k + t < K ? row[k + t] : (__bf16)0.0f;
    }
}
template <bool VEC> __device__ inline void load_x8(const float *row, int k, int K, bf16x8 (&p)[3])
{
    float v[8];
    if constexpr (VEC) {
        f32x4 a{}, b{};
        if (k < K) {
            a = *(const f32x4 *)(row + k);
            b = *(const f32x4 *)(row + k + 4);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) { v[t] = a[t]; v[t + 4] = b[t]; }
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = k + t < K ? row[k + t] : 0.0f;
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        unsigned short h, m, l;
        split3(v[t], h, m, l);
        p[0][t] = __builtin_bit_cast(__bf16, h);
        p[1][t] = __builtin_bit_cast(__bf16, m);
        p[2][t] = __builtin_bit_cast(__bf16, l);
    }
}

// Codes k .. k + 7 of a row, code t in bits 4t .. 4t + 3, zero past K.
template <bool VEC> __device__ inline unsigned load_c8(const uint8_t *row, int k, int K)
{
    unsigned w = 0;
    if constexpr (VEC) {
        if (k < K) w = *(const unsigned *)(row + k / 2);
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (k + 2 * t < K) w |= (unsigned)row[k / 2 + t] << (8 * t);
    }
    return w;
}

__device__ inline float int4_value(unsigned w, int t) { return (float)((int)(w << (28 - 4 * t)) >> 28); }

// One 16 x 16 tile of Y per workgroup, its K range dealt to the four waves and
// their sums added through LDS in wave order.  EXACT: int4 codes go to the
// matrix cores as they are, each group's sum is formed apart and multiplied by
// the group's scale (groups of 32 and more); else the dequantised fp32 weight is
// split into PW bf16 parts.
template <typename TX, typename TY, bool NF4, bool EXACT, int PW, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void int4_direct_kernel(I4Args a)
{
    constexpr int PX = sizeof(TX) == 4 ? 3 : 1;
    __shared__ float red[kWaves][256];
    __shared__ float lut[16];
    if (threadIdx.x < 16) lut[threadIdx.x] = kNF4[threadIdx.x];
    __syncthreads();
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, 16, grid_row(), rt)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int n = min(n0 + r, a.N - 1);
    const int64_t m = min(rt.r0 + r, rt.r1 - 1);
    const TX *x = (const TX *)a.X + m * a.ldx;
    const uint8_t *c = a.codes + (rt.e * a.N + n) * (int64_t)(a.K / 2);
    const float *sc = a.scales + (rt.e * a.N + n) * (int64_t)(a.K / a.G);
    f32x4 acc{};
    if constexpr (EXACT) {
        for (int g = wave; g < a.K / a.G; g += kWaves) {
            f32x4 part{};
            for (int k0 = g * a.G; k0 < (g + 1) * a.G; k0 += 32) {
                bf16x8 xp[PX], w;
                load_x8<VEC>(x, k0 + 8 * q, a.K, xp);
                const unsigned cw = load_c8<VEC>(c, k0 + 8 * q, a.K);
#pragma unroll
                for (int t = 0; t < 8; ++t) w[t] = (__bf16)int4_value(cw, t);
#pragma unroll
                for (int i = 0; i < PX; ++i) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xp[i], w, part, 0, 0, 0);
            }
            const float s = sc[g];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, part[i], acc[i]);
        }
    } else {
        for (int k0 = 32 * wave; k0 < a.K; k0 += 32 * kWaves) {
            bf16x8 xp[PX], wp[PW];
            load_x8<VEC>(x, k0 + 8 * q, a.K, xp);
            const unsigned cw = load_c8<VEC>(c, k0 + 8 * q, a.K);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int k = k0 + 8 * q + t;
                const float s = k < a.K ? sc[k / a.G] : 0.0f;
                const float v = (NF4 ? lut[(cw >> (4 * t)) & 15] : int4_value(cw, t)) * s;
                unsigned short p[3];
                split3(v, p[0], p[1], p[2]);
#pragma unroll
                for (int j = 0; j < PW; ++j) wp[j][t] = __builtin_bit_cast(__bf16, p[j]);
            }
            // parts i of X and j of W with i + j <= 2: what is left out is below 2^-24 of the product
#pragma unroll
            for (int i = 0; i < PX; ++i)
#pragma unroll
                for (int j = 0; j < PW; ++j)
                    if (i + j <= 2) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xp[i], wp[j], acc, 0, 0, 0);
        }
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
    if (row < rt.r1 && n0 + r < a.N) store_y((TY *)a.Y + row * a.ldy + n0 + r, v);
}

template <typename TX, typename TY, bool NF4, bool EXACT, int PW>
hipError_t launch_direct(const I4Args &a, bool vec, dim3 grid, hipStream_t s)
{
    if (vec) hipLaunchKernelGGL((int4_direct_kernel<TX, TY, NF4, EXACT, PW, true>), grid, dim3(64 * kWaves), 0, s, a);
    else hipLaunchKernelGGL((int4_direct_kernel<TX, TY, NF4, EXACT, PW, false>), grid, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- large tiles, bf16 X
// Eight codes of one dword as bf16, exactly: a byte holding a code in its high
// nibble is 16 code as a signed byte, one conversion per code; the factor 1/16
// goes with the scale.
__device__ inline bf16x8 bf16_of_int4(unsigned w)
{
    const unsigned lo = (w << 4) & 0xF0F0F0F0u, hi = w & 0xF0F0F0F0u;
    bf16x8 r;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        r[2 * t] = (__bf16)(float)(signed char)(lo >> (8 * t));
        r[2 * t + 1] = (__bf16)(float)(signed char)(hi >> (8 * t));
    }
    return r;
}

constexpr int kStage = 128;                 // k per stage

// WM x WN waves of PM x PN blocks of 16 x 16.
template <typename TY, int WM, int WN, int PM, int PN>
__global__ __launch_bounds__(64 * WM * WN, 2) void int4_tile_kernel(I4Args a, int64_t nt, int64_t mt)
{
    constexpr int NW = WM * WN, TM = 16 * WM * PM, TN = 16 * WN * PN, kRow = 2 * kStage;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    constexpr int kSlot = TM * kRow;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int64_t ti, tj;
    grouped_tile(blockIdx.x, nt, mt, ti, tj);
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, TM, ti, rt)) return;
    const int n0 = (int)tj * TN, K = a.K;
    const int mrows = (int)(rt.r1 - rt.r0);
    const uint8_t *xbase = (const uint8_t *)((const __bf16 *)a.X + rt.r0 * a.ldx);
    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 15, q = lane >> 4;

    // copy u: rows 4 wave + 4 NW u .. + 3, 256 bytes each; lane l takes position
    // l % 16 of row l / 16, chunk position ^ (row & 15).  The offsets are formed
    // at each copy: kept, they would not fit the registers beside the sums.
    constexpr int NC = TM / (4 * NW);
    static_assert((4 * NW) % 16 == 0, "row & 15 is the same for every u");
    int crow = 4 * wave + (lane >> 4);
    const unsigned ch = 16u * ((lane & 15) ^ (crow & 15));
    const unsigned ld2 = (unsigned)(2 * a.ldx);
    const unsigned lbase = lds_offset(lds);
    auto copy = [&](int b, int slot) {
        asm volatile("" : "+v"(crow));
#pragma unroll
        for (int u = 0; u < NC; ++u) {
            copy16_lds(xbase + 256 * b, (unsigned)min(crow + 4 * NW * u, mrows - 1) * ld2 + ch, lbase + slot * kSlot + 4 * (wave + NW * u) * kRow);
        }
    };
    const uint8_t *cbase = a.codes + (rt.e * a.N + n0) * (int64_t)(K / 2);
    const int nb = K / kStage;
    const float *sbase = a.scales + (rt.e * a.N + n0) * (int64_t)(K / a.G);
    const int nlast = a.N - n0 - 1;
    int nrow = 16 * PN * wn + r;
    u32x4 cn[PN];
    float sn[PN];
    auto load_w = [&](int b) {
        const uint8_t *cb = cbase + 64 * b;
        const float *sb = sbase + b;
        asm volatile("" : "+v"(nrow));
#pragma unroll
        for (int j = 0; j < PN; ++j) {
            const unsigned n = (unsigned)min(nrow + 16 * j, nlast);
            cn[j] = *(const u32x4 *)(cb + (n * (unsigned)(K / 2) + 16u * q));
            sn[j] = *(const float *)((const uint8_t *)sb + n * (unsigned)(4 * nb));
        }
    };
    f32x4 acc[PM][PN];
#pragma unroll
    for (int i = 0; i < PM; ++i)
#pragma unroll
        for (int j = 0; j < PN; ++j) acc[i][j] = f32x4{};
    copy(0, 0);
    load_w(0);
    const int rx = r * kRow;
    for (int b = 0; b < nb; ++b) {
        const int slot = b & 1;
        publish();
        bf16x8 w[PN][4];
        float s[PN];
#pragma unroll
        for (int j = 0; j < PN; ++j) {
#pragma unroll
            for (int h = 0; h < 4; ++h) w[j][h] = bf16_of_int4(cn[j][h]);
            s[j] = sn[j] * 0.0625f;
        }
        if (b + 1 < nb) {
            copy(b + 1, slot ^ 1);
            load_w(b + 1);
        }
        const uint8_t *xs = lds + slot * kSlot + 16 * PM * wm * kRow + rx;
#pragma unroll
        for (int i = 0; i < PM; ++i) {
            bf16x8 x[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) x[h] = *(const bf16x8 *)(xs + 16 * i * kRow + 16 * ((4 * q + h) ^ r));
#pragma unroll
            for (int j0 = 0; j0 < PN; j0 += 2) {
                f32x4 part[2] = {};
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        part[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[h], w[j0 + j][h], part[j], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[i][j0 + j][t] = fmaf(s[j0 + j], part[j][t], acc[i][j0 + j][t]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PM; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t row = rt.r0 + 16 * (PM * wm + i) + 4 * q + t;
            if (row >= rt.r1) continue;
            TY *y = (TY *)a.Y + row * a.ldy;
#pragma unroll
            for (int j = 0; j < PN; ++j) {
                const int n = n0 + 16 * (PN * wn + j) + r;
                if (n < a.N) store_y(y + n, acc[i][j][t]);
            }
        }
}

template <typename TY, int WM, int WN, int PM, int PN> hipError_t launch_tile(const I4Args &a, hipStream_t s)
{
    constexpr int TM = 16 * WM * PM, TN = 16 * WN * PN;
    constexpr size_t lds = 2 * (size_t)TM * 2 * kStage;
    const auto kernel = int4_tile_kernel<TY, WM, WN, PM, PN>;
    static const bool lds_ok = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) == hipSuccess;
    if (!lds_ok) return hipErrorInvalidConfiguration;
    const int64_t nt = (a.N + TN - 1) / TN, mt = row_tiles(a.offsets != nullptr, a.E, a.M, TM);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(nt * mt)), dim3(64 * WM * WN), lds, s, a, nt, mt);
    return hipGetLastError();
}

template <typename TX, typename TY> hipError_t launch_int4(I4Args a, bool nf4, hipStream_t s)
{
    if constexpr (sizeof(TX) == 2) {
        if (a.M > 64 && !nf4 && a.G == 128 && a.ldx % 8 == 0 && a.ldx <= (1 << 22) && ((uintptr_t)a.X & 15) == 0 && ((uintptr_t)a.codes & 15) == 0)
            return launch_tile<TY, 1, 4, 8, 4>(a, s);
    }
    const dim3 grid = tile_grid((a.N + 15) / 16, row_tiles(a.offsets != nullptr, a.E, a.M, 16));
    const bool vec = a.K % 8 == 0 && ((uintptr_t)a.X & 15) == 0 && (a.ldx * sizeof(TX)) % 16 == 0 &&
                     ((uintptr_t)a.codes & 3) == 0;
    if (nf4) return launch_direct<TX, TY, true, false, 3>(a, vec, grid, s);
    if (a.G >= 32) return launch_direct<TX, TY, false, true, 1>(a, vec, grid, s);
    return launch_direct<TX, TY, false, false, 3>(a, vec, grid, s);
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
    if (M > INT32_MAX || N > (1 << 24) || K > (1 << 24)) return set_error(GQ_ERR_INVALID_ARG, "size too large");
    if (M == 0) return set_error(GQ_OK, "");
    if (!Y || !X || !codes || !scales) return set_error(GQ_ERR_INVALID_ARG, "null required pointer");
    I4Args a{};
    a.Y = Y; a.X = X; a.codes = codes; a.scales = scales; a.offsets = offsets;
    a.M = M; a.ldx = ldx; a.ldy = ldy; a.E = E;
    a.N = (int)N; a.K = (int)K; a.G = (int)group;
    const bool nf4 = flags & GQ_NF4;
    hipError_t e;
    if (x_dtype == GQ_F32)
        e = y_dtype == GQ_F32 ? launch_int4<float, float>(a, nf4, stream) : launch_int4<float, __bf16>(a, nf4, stream);
    else
        e = y_dtype == GQ_F32 ? launch_int4<__bf16, float>(a, nf4, stream) : launch_int4<__bf16, __bf16>(a, nf4, stream);
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
