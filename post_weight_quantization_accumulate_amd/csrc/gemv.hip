// gemv.hip -- pack products of one or two rows: a decoding step, where reading
// the pack is the work.
//
// A lane owns 32 consecutive k for the whole call: their x stay in its registers
// as fp32, and for each column n of Y (row n of the pack) it loads its 16 bytes of
// int4 codes (32 of e4m3), neighbouring lanes neighbouring bytes, so every load of
// a wave is one contiguous run.  A workgroup is the waves of one row of the pack
// and takes COLS columns, all their loads issued at once.  All arithmetic is fp32
// (codes, NF4 levels and e4m3 values are exact in it); a lane's 32 products lie
// within one group and are scaled once.  The four sums of a wave are reduced
// together: two of them change halves (then quarters) with one swap, so it takes
// 10 instructions, not 24.
// The matrix cores would need each lane's loads 16 rows apart and x loaded again
// for every 16 columns.  Bound by memory: 1 x 5120 x 17408 e4m3 takes 21 us (4.2
// TB/s, a large copy reaches 5.2), 1 x 10240 x 5120 int4 8.7 us (3.2 TB/s; the
// arithmetic, 2.4 instructions per code, takes about 3 of them).
#include "gemv.h"

namespace gq {
namespace {

constexpr int SEG = 32;                 // k per lane

__device__ inline float swap_add32(float a, float b)
{
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 v = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(v[0]) + __uint_as_float(v[1]);
}
__device__ inline float swap_add16(float a, float b)
{
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 v = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(v[0]) + __uint_as_float(v[1]);
}
template <int N> __device__ inline float add_ror(float v)
{
    return v + __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0x120 + N, 0xF, 0xF, true));
}
// Sums of v[0..3] over the wave; lanes 16 p .. 16 p + 15 get that of v[kSumOf(p)].
__device__ inline float sum4(const float (&v)[4])
{
    float s = swap_add16(swap_add32(v[0], v[1]), swap_add32(v[2], v[3]));
    s = add_ror<8>(s);
    s = add_ror<4>(s);
    s = add_ror<2>(s);
    return add_ror<1>(s);
}
__device__ inline int sum_of(int p) { return (p >> 1) | ((p & 1) << 1); }

// The 32 products of one column and MR rows.
template <int KIND, int MR>
__device__ inline void dot32(const u32x4 (&c)[KIND == GEMV_FP8 ? 2 : 1], const float *lut, const float (&x)[MR][SEG], float (&dot)[MR])
{
#pragma unroll
    for (int m = 0; m < MR; ++m) dot[m] = 0.0f;
    if constexpr (KIND == GEMV_FP8) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const int w = (int)c[d >> 2][d & 3];
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                dot[m] = fmaf(lo[0], x[m][4 * d], dot[m]);
                dot[m] = fmaf(lo[1], x[m][4 * d + 1], dot[m]);
                dot[m] = fmaf(hi[0], x[m][4 * d + 2], dot[m]);
                dot[m] = fmaf(hi[1], x[m][4 * d + 3], dot[m]);
            }
        }
    } else {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const unsigned w = c[0][d];
            const unsigned lo = (w << 4) & 0xF0F0F0F0u, hi = w & 0xF0F0F0F0u;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float v0, v1;
                if constexpr (KIND == GEMV_INT4) {      // 16 times the code
                    v0 = (float)(signed char)(lo >> (8 * t));
                    v1 = (float)(signed char)(hi >> (8 * t));
                } else {                                // byte offset 4 code of the level
                    v0 = *(const float *)((const char *)lut + ((w << 2 >> (8 * t)) & 0x3C));
                    v1 = *(const float *)((const char *)lut + ((w >> (8 * t + 2)) & 0x3C));
                }
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    dot[m] = fmaf(v0, x[m][8 * d + 2 * t], dot[m]);
                    dot[m] = fmaf(v1, x[m][8 * d + 2 * t + 1], dot[m]);
                }
            }
        }
    }
}

__device__ inline void load_x32(const __bf16 *p, float (&x)[SEG])
{
    bf16x8 v[4];
    __builtin_memcpy(v, p, sizeof v);
#pragma unroll
    for (int t = 0; t < SEG; ++t) x[t] = (float)v[t / 8][t % 8];
}
__device__ inline void load_x32(const float *p, float (&x)[SEG]) { __builtin_memcpy(x, p, sizeof x); }

template <int KIND, typename TX, int MR, int COLS, int MAXT>
__global__ __launch_bounds__(MAXT) void gemv_kernel(GemvArgs a)
{
    constexpr int NL = KIND == GEMV_FP8 ? 2 : 1, CB = 16 * NL;     // 16-byte loads and bytes per lane and column
    __shared__ float part[MAXT / 64][MR][COLS];
    __shared__ float lut[16];
    if constexpr (KIND == GEMV_NF4) {
        if (threadIdx.x < 16) lut[threadIdx.x] = kNF4[threadIdx.x];
        __syncthreads();
    }
    RowTile rt;
    if (!row_tile(a.offsets, (int)a.E, a.M, MR, grid_row(), rt)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), WR = (int)(blockDim.x >> 6);
    const int n0 = blockIdx.x * COLS, segs = (a.K + SEG - 1) / SEG;
    const int sg = min(wave * 64 + lane, segs - 1);
    // a last segment that is not whole (e4m3 only) ends with the row; the x of what
    // belongs to the lane before it are zero
    const int k0 = min(sg * SEG, a.K - SEG), over = sg * SEG - k0;
    const bool in = wave * 64 + lane < segs;                         // lanes past the row add zeros
    const int64_t rowb = KIND == GEMV_FP8 ? a.K : a.K / 2;
    const int nsc = KIND == GEMV_FP8 ? (a.K + 127) / 128 : a.K / a.G;      // scales per row
    const int lg = __builtin_ctz(a.G);
    const uint8_t *cb = a.codes + rt.e * a.N * rowb + (int64_t)k0 * CB / SEG;
    const float *sb = a.scales + rt.e * (KIND == GEMV_FP8 ? (a.N + 127) / 128 : a.N) * (int64_t)nsc + ((sg * SEG) >> lg);
    u32x4 c[COLS][NL];
    float sc[COLS];
#pragma unroll
    for (int b = 0; b < COLS; ++b) {
        const int n = min(n0 + b, a.N - 1);
#pragma unroll
        for (int l = 0; l < NL; ++l) __builtin_memcpy(&c[b][l], cb + n * rowb + 16 * l, 16);
        sc[b] = sb[(KIND == GEMV_FP8 ? n / 128 : n) * (int64_t)nsc];
    }
    float x[MR][SEG];
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        const int64_t row = min(rt.r0 + m, rt.r1 - 1);
        if constexpr (KIND == GEMV_FP8) {
            u32x4 v[2];
            __builtin_memcpy(v, (const uint8_t *)a.X + row * a.K + k0, 32);
            const float s = a.xs[row * nsc + (sg * SEG >> 7)];
            typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[d >> 2][d & 3], false);
                const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[d >> 2][d & 3], true);
                x[m][4 * d] = lo[0] * s; x[m][4 * d + 1] = lo[1] * s; x[m][4 * d + 2] = hi[0] * s; x[m][4 * d + 3] = hi[1] * s;
            }
        } else {
            load_x32((const TX *)a.X + row * a.ldx + sg * SEG, x[m]);
        }
#pragma unroll
        for (int t = 0; t < SEG; ++t) x[m][t] = in && (KIND != GEMV_FP8 || t >= over) ? x[m][t] : 0.0f;
    }
#pragma unroll
    for (int b0 = 0; b0 < COLS; b0 += 4) {
        float d[MR][4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float dot[MR];
            dot32<KIND, MR>(c[b0 + b], lut, x, dot);
            const float s = in ? (KIND == GEMV_INT4 ? sc[b0 + b] * 0.0625f : sc[b0 + b]) : 0.0f;
#pragma unroll
            for (int m = 0; m < MR; ++m) d[m][b] = s * dot[m];
            // one column at a time: put off to where its sum is needed, a row's
            // products would keep every converted value of four columns alive
            if constexpr (MR > 1) {
#pragma unroll
                for (int m = 0; m < MR; ++m) asm volatile("" : "+v"(d[m][b]));
            }
        }
        float v[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) v[m] = sum4(d[m]);
        if ((lane & 15) == 0) {
#pragma unroll
            for (int m = 0; m < MR; ++m) part[wave][m][b0 + sum_of(lane >> 4)] = v[m];
        }
    }
    __syncthreads();
    if (threadIdx.x < MR * COLS) {
        const int m = threadIdx.x / COLS, b = threadIdx.x % COLS;
        float v = part[0][m][b];
        for (int w = 1; w < WR; ++w) v += part[w][m][b];
        const int64_t row = rt.r0 + m;
        if (row < rt.r1 && n0 + b < a.N) {
            if (a.y_bf16) ((__bf16 *)a.Y)[row * a.ldy + n0 + b] = (__bf16)v;
            else ((float *)a.Y)[row * a.ldy + n0 + b] = v;
        }
    }
}

// Waves to a row of the pack.
constexpr int row_waves(int K) { return ((K + SEG - 1) / SEG + 63) / 64; }

// Waves of a workgroup that leave each the registers its x need.
constexpr int max_waves(int mr) { return mr == 1 ? 16 : 10; }

template <int KIND, typename TX, int MR, int COLS> hipError_t launch_cols(const GemvArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((gemv_kernel<KIND, TX, MR, COLS, 64 * max_waves(MR)>),
                       tile_grid((a.N + COLS - 1) / COLS, row_tiles(a.offsets != nullptr, a.E, a.M, MR)),
                       dim3(64 * row_waves(a.K)), 0, s, a);
    return hipGetLastError();
}
// Eight columns share each x and are the rule.  Four leave fewer CUs without work
// where there are fewer than two workgroups to a CU (1 x 1024 x 5120: 3.3 against
// 4.0 us), or where those of eight would fill their last round badly (1 x 5120 x
// 17408 int4, 640 workgroups of which 512 run at a time: 14.9 against 19.4 us; 1 x
// 8192 x 28672, four full rounds: 38.9 against 33.6 us).
template <int KIND, typename TX, int MR> hipError_t launch_rows(const GemvArgs &a, hipStream_t s)
{
    constexpr int kWaves = MR == 2 ? 12 : KIND == GEMV_INT4 ? 20 : 16;      // to a CU, by the registers
    const int64_t wgs = (a.N + 7) / 8 * row_tiles(a.offsets != nullptr, a.E, a.M, MR);
    const int64_t slots = 256 * (row_waves(a.K) < kWaves ? kWaves / row_waves(a.K) : 1);
    const bool badly = wgs > slots && 4 * wgs < 3 * slots * ((wgs + slots - 1) / slots);
    return wgs < 512 || badly ? launch_cols<KIND, TX, MR, 4>(a, s) : launch_cols<KIND, TX, MR, 8>(a, s);
}

template <int KIND, typename TX> hipError_t by_rows(const GemvArgs &a, int rows, hipStream_t s)
{
    if (rows <= 1) return launch_rows<KIND, TX, 1>(a, s);
    return launch_rows<KIND, TX, 2>(a, s);
}

}  // namespace

bool gemv_ok(const GemvArgs &a, int kind, int rows)
{
    return rows <= kGemvMaxRows && a.G >= SEG && row_waves(a.K) <= max_waves(rows) &&
           (kind == GEMV_FP8 ? a.K >= SEG : a.K % SEG == 0);
}

hipError_t launch_gemv(const GemvArgs &a, int kind, int rows, hipStream_t s)
{
    if (kind == GEMV_FP8) return by_rows<GEMV_FP8, uint8_t>(a, rows, s);
    if (kind == GEMV_NF4) return a.x_bf16 ? by_rows<GEMV_NF4, __bf16>(a, rows, s) : by_rows<GEMV_NF4, float>(a, rows, s);
    return a.x_bf16 ? by_rows<GEMV_INT4, __bf16>(a, rows, s) : by_rows<GEMV_INT4, float>(a, rows, s);
}

}  // namespace gq
