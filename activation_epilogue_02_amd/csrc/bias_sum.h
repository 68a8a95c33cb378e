// bias_sum.h -- the bias gradient from its partial sums.
#pragma once

#include "ge_device.h"

namespace ge {

// out[j] = sum over t < parts of partial[t][j], rows of `len`, in a fixed order:
// workgroup `block` takes 32 entries, eight groups of 32 lanes every eighth
// partial each, then the groups in order (one lane per entry over all
// partials: 40 us for 128 partials of 4096 entries, as long as writing dP).
// red: 8 x 33 floats of LDS.  parts = 0 writes zeros.  Threads past 256 only
// meet the barrier.
constexpr int kSumCols = 32, kSumGroups = 8;
template <int DT>
__device__ __forceinline__ void sum_partials(const float* partial, int parts, int len, void* out, int block, int tid,
                                             float (*red)[kSumCols + 1]) {
    const int c = tid & 31, g = tid >> 5;
    const int64_t j = (int64_t)block * kSumCols + c;
    if (g < kSumGroups) {
        float v = 0.0f;
        if (j < len) {
#pragma unroll 8
            for (int t = g; t < parts; t += kSumGroups) v += partial[(int64_t)t * len + j];
        }
        red[g][c] = v;
    }
    __syncthreads();
    if (g == 0 && j < len) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kSumGroups; ++i) s += red[i][c];
        store_one<DT>(out, j, s);
    }
}

}  // namespace ge
