// matmul.h -- shared parts of the pack products (int4mm.hip, fp8.hip): the row
// tile of a workgroup with and without experts, bf16 parts of fp32 values, and
// rounding to the output type.
#pragma once

#include <hip/hip_runtime.h>
#include <atomic>
#include <stdint.h>

#include "gq_internal.h"

namespace gq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Rows r0 .. r1 - 1 of X and Y that a workgroup takes, and the pack they go with.
struct RowTile {
    int64_t r0, r1;
    int64_t e;
};

// Row tile number `t` of tiles of TM rows.  Without offsets the rows are
// 0 .. M - 1 of pack 0.  With offsets (E + 1 device ints) expert e has the rows
// offsets[e] .. offsets[e + 1] - 1, in tiles of its own.  The tiles are counted
// 64 experts at a time, one per lane, with a wave prefix sum, so no host copy of
// the offsets is needed; every wave of a workgroup finds the same answer by
// itself.  The offsets are clamped to 0 <= offsets[e] <= offsets[e + 1] <= M, so
// that no value of theirs leads outside X and Y.  False: no such tile.
__device__ inline bool row_tile(const int *offsets, int E, int64_t M, int TM, int64_t t, RowTile &out)
{
    if (!offsets) {
        out.r0 = t * TM;
        out.r1 = min(out.r0 + TM, M);
        out.e = 0;
        return out.r0 < M;
    }
    const int lane = threadIdx.x & 63;
    int want = (int)t;
    for (int base = 0; base < E; base += 64) {
        int lo = 0, hi = 0;
        if (base + lane < E) {
            lo = min(max(offsets[base + lane], 0), (int)M);
            hi = min(max(offsets[base + lane + 1], lo), (int)M);
        }
        const int nt = (hi - lo) / TM + ((hi - lo) % TM != 0);
        int inc = nt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(inc, d);
            if (lane >= d) inc += v;
        }
        const int total = __builtin_amdgcn_readlane(inc, 63);
        if (want < total) {
            const int f = __builtin_ctzll(__ballot(inc > want));
            const int first = __builtin_amdgcn_readlane(inc - nt, f);
            const int elo = __builtin_amdgcn_readlane(lo, f), ehi = __builtin_amdgcn_readlane(hi, f);
            out.r0 = elo + (int64_t)(want - first) * TM;
            out.r1 = min(out.r0 + TM, (int64_t)ehi);
            out.e = base + f;
            return true;
        }
        want -= total;
    }
    return false;
}

// Lets Kernel use `bytes` of dynamic LDS on the current device (asked for once per
// device).
template <auto Kernel> hipError_t allow_lds(size_t bytes)
{
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
    const hipError_t f = hipFuncSetAttribute((const void *)Kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (f == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return f;
}

// A launch holds fewer than 2^32 threads in a dimension.
inline bool grid_fits(int64_t blocks, int threads) { return blocks * threads < (int64_t)1 << 32; }

// An upper bound of the number of row tiles: with experts every tile holds a
// row and every expert adds at most one partly filled tile.
inline int64_t row_tiles(bool experts, int64_t E, int64_t M, int64_t TM)
{
    if (!experts) return (M + TM - 1) / TM;
    const int64_t n = M / TM + E;
    return n < M ? n : M;
}

// A grid of nt column tiles (x) by mt row tiles (y and z): row tile
// blockIdx.z * kGridRows + blockIdx.y.
constexpr int64_t kGridRows = 32768;
inline dim3 tile_grid(int64_t nt, int64_t mt)
{
    const int64_t z = (mt + kGridRows - 1) / kGridRows;
    return dim3((unsigned)nt, (unsigned)(z > 1 ? kGridRows : mt), (unsigned)z);
}
__device__ inline int64_t grid_row() { return (int64_t)blockIdx.z * kGridRows + blockIdx.y; }

// Workgroup `w` of nt x mt tiles: each XCD gets a contiguous run of tiles (see
// xcd_order), which walk the grid in groups of kGroupRows row tiles, so that the
// tiles that run together on one XCD share their operands in its L2.
constexpr int64_t kGroupRows = 8;
__device__ inline void grouped_tile(int64_t w, int64_t nt, int64_t mt, int64_t &ti, int64_t &tj)
{
    const int64_t id = xcd_order(w, nt * mt);
    const int64_t g = id / (kGroupRows * nt), first = g * kGroupRows;
    const int64_t rows = min(kGroupRows, mt - first), in = id - first * nt;
    ti = first + in % rows;
    tj = in / rows;
}

// 64 lanes x 16 (or 4) bytes from base + off (off per lane) to LDS at l + 16
// (4) lane, past the registers.  Inline asm, so that the compiler does not wait
// for every copy before any LDS read: the caller waits with wait_copies before
// the barrier that publishes them.  M0 is set right before each copy and used
// by nothing else.
__device__ inline void copy16_lds(const void *base, unsigned off, unsigned l)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(l) : "memory");
}
__device__ inline void copy4_lds(const void *base, unsigned off, unsigned l)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(l) : "memory");
}
// Waits until at most N of this wave's memory instructions are under way; they
// end in order.
template <int N = 0> __device__ inline void wait_copies()
{
    static_assert(N >= 0 && N < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Waits for this wave's LDS reads (and writes): before a copy may overwrite them.
__device__ inline void wait_lds()
{
    __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0), the other counters at their maxima
    asm volatile("" ::: "memory");
}

// Runs the units u0 .. u1 - 1 of a wave through two slots of its own part of LDS:
// issue(u, slot) starts the LOADS copies of a unit, use(u, slot) consumes it while
// the next unit's are under way.  Only copies (which the compiler does not know
// of) load from memory in here, so that the waits are these alone.
template <int LOADS, typename Issue, typename Use> __device__ inline void ring(int u0, int u1, Issue issue, Use use)
{
    if (u0 < u1) issue(u0, 0);
    int slot = 0;
    for (int u = u0; u < u1; ++u) {
        if (u + 1 < u1) {
            wait_lds();
            issue(u + 1, slot ^ 1);
            wait_copies<LOADS>();
        } else {
            wait_copies<0>();
        }
        use(u, slot);
        slot ^= 1;
    }
}

__device__ inline void publish()
{
    wait_copies();
    __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0): this wave's LDS writes
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
__device__ inline unsigned lds_offset(const void *p)
{
    return (unsigned)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// 16 bytes from p, of which only the first n are the caller's (the rest zero);
// p may be unaligned.
__device__ inline u32x4 load16(const uint8_t *p, int n)
{
    u32x4 v{};
    if (n >= 16) __builtin_memcpy(&v, p, 16);
    else
        for (int i = 0; i < n; ++i) v[i >> 2] |= (unsigned)p[i] << (8 * (i & 3));
    return v;
}

__device__ inline void store_y(float *p, float v) { *p = v; }
__device__ inline void store_y(__bf16 *p, float v) { *p = (__bf16)v; }

}  // namespace gq
