// norm_params.h -- argument block and launch interface of the RMS-norm
// kernels, shared by the front end (norm_api.cpp) and norm_kernel.hip.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/ge_rms_norm.h"

namespace ge {

struct NormArgs {
    const void* x;       // forward: input; backward: h
    const void* res;     // forward: residual or NULL
    const void* gamma;
    void* h;             // forward: the rounded sum, or NULL
    void* y;
    void* scales;        // E4M3_ROW: fp32 per row; MX: E8M0 bytes
    float* rstd;         // forward: output or NULL; backward: input
    const void* dy;
    const void* dh;      // or NULL
    void* dx;
    void* dgamma;        // or NULL
    float* partial;      // backward: blocks x cols fp32
    int32_t rows, cols;
    int32_t blocks;      // workgroups of the launch
    int32_t lds;         // MX: bytes per row of scales
    int64_t ld, ldy;
    float eps, inv_cols;
};

// Threads per row and 16-byte chunks per thread of a launch; chunks == 0 is
// the kernel for rows that no register shape holds.
struct NormShape {
    int32_t threads, chunks;
};
constexpr NormShape kNormFwd[] = {{64, 1}, {64, 2}, {256, 1}, {256, 2}, {256, 3}, {256, 4}, {1024, 2}, {1024, 4}};
constexpr NormShape kNormBwd[] = {{64, 1}, {64, 2}, {256, 1}, {256, 2}, {256, 3}, {512, 2}, {512, 3}, {1024, 2}, {1024, 4}};
constexpr NormShape kNormLong = {1024, 0};

int launch_norm_forward(int type, int out, NormShape s, const NormArgs& a, void* stream);
int launch_norm_backward(int type, NormShape s, const NormArgs& a, void* stream);
// dgamma from the partial sums (a.blocks of them; 0 writes zeros)
int launch_norm_dgamma(int type, const NormArgs& a, void* stream);

}  // namespace ge
