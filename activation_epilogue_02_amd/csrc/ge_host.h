// ge_host.h -- host helpers of the C-ABI front ends (api.cpp, norm_api.cpp).
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

#include "../../include/gemm_epilog.h"

namespace ge {

inline int elem_size(int t) {
    switch (t) {
    case GE_F32: return 4;
    case GE_F16: return 2;
    case GE_BF16: return 2;
    case GE_F8_E4M3: return 1;
    case GE_MXF8_E4M3: return 1;
    }
    return 0;
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// GE_LOG=1 in the environment: every successful plan prints its
// description (path, tile, grid, split, workspace) to stderr.
inline bool plan_log() {
    const char* e = getenv("GE_LOG");
    return e && e[0] == '1';
}

// GE_TEST_FAIL_LAUNCH=1: a call that passed its checks reports GE_ERR_HIP
// instead of launching (error-path tests).
inline bool test_fail_launch() {
    const char* e = getenv("GE_TEST_FAIL_LAUNCH");
    return e && e[0] == '1';
}

}  // namespace ge
