// gemv.h -- pack products of a few rows each (gemv.hip).
#pragma once

#include "gq_internal.h"
#include "matmul.h"

namespace gq {

enum : int { GEMV_INT4 = 0, GEMV_NF4 = 1, GEMV_FP8 = 2 };

struct GemvArgs {
    void *Y;
    const void *X;              // rows of X (bf16 or fp32), or e4m3 codes
    const float *xs;            // e4m3: X's scales
    const uint8_t *codes;
    const float *scales;
    const int *offsets;
    int64_t M, ldx, ldy, E;
    int N, K, G;                // G: columns per scale (fp8: 128)
    bool y_bf16, x_bf16;
};

// Rows per tile above which the matrix cores win.
constexpr int kGemvMaxRows = 2;
// True if the kernel takes these sizes: at least one piece of 32 codes to a row
// (int4: whole pieces), scales no finer than that, at most 16 waves to a row.
bool gemv_ok(const GemvArgs &a, int kind, int rows);
hipError_t launch_gemv(const GemvArgs &a, int kind, int rows, hipStream_t s);

}  // namespace gq
