// grad_params.h -- argument block and launch interface of grad_kernel.hip.
#pragma once

#include <stdint.h>

namespace ge {

struct GradArgs {
    const void* src;    // rows x cols, row stride ld
    const void* aux;    // MASK: words, GELU: pre-activation; row stride ldaux
    void* dst;          // dP (MASK, GELU), row stride ldd, or NULL
    void* dst_t;        // the transpose, cols x rows, row stride ldt, or NULL
    float* partial;     // bias gradient: COL [row tile][col], ROW [column tile][row]; or NULL
    int32_t rows, cols;
    int32_t axis, ldaux;
    int64_t ld, ldd, ldt;
};

// COPY: transpose only.  PLAIN: dP = dD.
enum GradKind { GRAD_COPY = 0, GRAD_PLAIN = 1, GRAD_MASK = 2, GRAD_GELU = 3 };
constexpr int kGradTile = 64;

int launch_grad_prepare(int type, int kind, const GradArgs& a, void* stream);
// out[j] = sum over t < parts of partial[t][j], j < len (parts = 0: zeros)
int launch_grad_bias(int type, const float* partial, int parts, int len, void* out, void* stream);

}  // namespace ge
