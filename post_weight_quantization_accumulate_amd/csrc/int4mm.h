// int4mm.h -- shared parts of the int4 / NF4 pack products: the arguments, codes
// to bf16, activations to bf16 parts.
#pragma once

#include "gq_internal.h"
#include "matmul.h"

namespace gq {

struct I4Args {
    void *Y;
    const void *X;
    const uint8_t *codes;
    const float *scales;
    const int *offsets;
    int64_t M, ldx, ldy, E;
    int N, K, G;
    bool y_bf16;
};

// How a pack's codes enter the bf16 matrix cores.
//   W_INT4  the code itself, exactly, in one bf16;
//   W_NF4   its level (fp32) as two or three bf16 parts: two (16 leading bits,
//           2^-16 off at most) where the result is rounded to bf16 anyway.
enum : int { W_INT4 = 0, W_NF4_2 = 2, W_NF4_3 = 3 };
template <int WM> struct WParts { static constexpr int n = WM == W_INT4 ? 1 : WM; };

// fp32 as N bf16 parts of its sign, 8 leading bits of what is left each, by
// truncation: three parts are exact.  No part but the last takes all that is left,
// so none is 0 unless the weight is: an infinite x then gives an infinity, not
// infinity times 0.
template <int N> __device__ inline void weight_parts(float v, unsigned short (&p)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        unsigned b = __float_as_uint(v) & 0xFFFF0000u;
        if (j + 1 < N && v != 0.0f && __uint_as_float(b) == v) b -= 0x10000u;
        p[j] = (unsigned short)(b >> 16);
        v -= __uint_as_float(b);
    }
}

// The bf16 parts of the NF4 levels of a byte's two codes, the low nibble's in the
// low half: an LDS table that turns a byte into operand dwords at one read, where
// a table of single levels takes two reads and a byte permute per part (64 x
// 10240 x 5120, groups of 64: 68 -> 39 us), though its reads meet in a bank more often.
struct Nf4Table {
    uint2 hm[256];              // first and second parts
    unsigned l[256];            // third parts
    template <int N> __device__ void fill()
    {
        for (int i = threadIdx.x; i < 256; i += blockDim.x) {
            unsigned short p[N], o[N];
            weight_parts(kNF4[i & 15], p);
            weight_parts(kNF4[i >> 4], o);
            hm[i] = make_uint2(p[0] | (unsigned)o[0] << 16, p[1] | (unsigned)o[1] << 16);
            if constexpr (N == 3) l[i] = p[2] | (unsigned)o[2] << 16;
        }
    }
};

// Eight codes of one dword (code t in bits 4t ..) as the PW bf16 parts of
// kCodeScale times their values.  int4: a byte holding a code in its high nibble
// is 16 times the code as a signed byte, one conversion each; the factor is taken
// out of the scale.
template <int WM> struct CodeScale { static constexpr float v = WM == W_INT4 ? 16.0f : 1.0f; };
template <int WM> __device__ inline void code_parts(unsigned w, const Nf4Table &tab, bf16x8 (&p)[WParts<WM>::n])
{
    if constexpr (WM == W_INT4) {
        const unsigned lo = (w << 4) & 0xF0F0F0F0u, hi = w & 0xF0F0F0F0u;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            p[0][2 * t] = (__bf16)(float)(signed char)(lo >> (8 * t));
            p[0][2 * t + 1] = (__bf16)(float)(signed char)(hi >> (8 * t));
        }
    } else {
        u32x4 o[WM];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const unsigned c = (w >> (8 * t)) & 255;
            const uint2 v = tab.hm[c];
            o[0][t] = v.x;
            o[1][t] = v.y;
            if constexpr (WM == W_NF4_3) o[2][t] = tab.l[c];
        }
#pragma unroll
        for (int j = 0; j < WM; ++j) p[j] = __builtin_bit_cast(bf16x8, o[j]);
    }
}

// Transposes a 4 x 4 array of dwords whose column is the lane's group of 16
// (q = lane / 16) and whose row is the register: d[h] of group q becomes d[q] of
// group h.  Loads want 16 consecutive bytes of codes per lane, and a matrix
// instruction that has to stay within a group wants 32 consecutive k over the four
// groups of lanes: this turns one into the other.
__device__ inline void transpose4(unsigned (&d)[4])
{
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    u32x2 a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    u32x2 b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    u32x2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    u32x2 e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = c[0]; d[1] = c[1]; d[2] = e[0]; d[3] = e[1];
}

// Eight consecutive elements of X from memory or LDS (16-byte pieces) as bf16 parts.
template <typename TX> struct XParts { static constexpr int n = sizeof(TX) == 4 ? 3 : 1; };
__device__ inline void x_parts(const __bf16 *p0, const __bf16 *, bf16x8 (&p)[1]) { p[0] = *(const bf16x8 *)p0; }
// fp32 as three parts of 8 leading bits by truncation, exactly: an infinity stays
// in the first part alone; a NaN, whose differences are NaN, needs no care.
__device__ inline void x_parts(f32x4 a, f32x4 b, bf16x8 (&p)[3])
{
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    unsigned d[3][8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        d[0][t] = __float_as_uint(v[t]);
        const float r = __builtin_isinf(v[t]) ? 0.0f : v[t] - __uint_as_float(d[0][t] & 0xFFFF0000u);
        d[1][t] = __float_as_uint(r);
        d[2][t] = __float_as_uint(r - __uint_as_float(d[1][t] & 0xFFFF0000u));
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        u32x4 o;
#pragma unroll
        for (int t = 0; t < 4; ++t) o[t] = __builtin_amdgcn_perm(d[j][2 * t + 1], d[j][2 * t], 0x07060302u);
        p[j] = __builtin_bit_cast(bf16x8, o);
    }
}
// p0, p1: the two 16-byte halves (4 elements each)
__device__ inline void x_parts(const float *p0, const float *p1, bf16x8 (&p)[3])
{
    x_parts(*(const f32x4 *)p0, *(const f32x4 *)p1, p);
}

// part += sum over the parts i of X and j of W with i + j <= 2: what is left out
// is below 2^-24 of each product.
template <int PX, int PW> __device__ inline f32x4 mma_parts(const bf16x8 (&x)[PX], const bf16x8 (&w)[PW], f32x4 part)
{
#pragma unroll
    for (int i = 0; i < PX; ++i)
#pragma unroll
        for (int j = 0; j < PW; ++j)
            if (i + j <= 2) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], w[j], part, 0, 0, 0);
    return part;
}

__device__ inline void store_row(const I4Args &a, int64_t row, int n, float v)
{
    if (a.y_bf16) ((__bf16 *)a.Y)[row * a.ldy + n] = (__bf16)v;
    else ((float *)a.Y)[row * a.ldy + n] = v;
}

// Groups of 32 and more, any M, K, strides and alignment (int4_tile.hip), and the
// same for few rows, aligned to 16 bytes (int4_skinny.hip).  The costs are
// estimates of the time in us of bf16 rows at K = 5120, for choosing between the
// tile shapes and the two; they grow alike with K and the types.
double int4_tile_cost(const I4Args &a, bool x_bf16, bool nf4, int *shape);
hipError_t launch_int4_tile(const I4Args &a, bool x_bf16, bool nf4, int shape, hipStream_t s);
double int4_skinny_cost(const I4Args &a, int *shape);
hipError_t launch_int4_skinny(const I4Args &a, bool x_bf16, bool nf4, int shape, hipStream_t s);

}  // namespace gq
