// res_epilogue.h -- the residual product's epilogue on a tile's fp32
// accumulators: D = R + act(s * row_scale[i] * col_scale[j] * C + bias), with
// the ReLU sign mask or the pre-activation as an optional second output.
//
// The residual is added after the activation, so a block's output leaves with
// the residual stream already in it and R is read where D is written, once.
// Each kind is compiled as a copy of its own, picked once per tile: one body
// that tests the kind per element is several times as much code, fetched cold
// at the end of every tile.  Column groups are the outer loop, so that the
// column scales and the bias are loaded once per group and reused by the
// lane's FM rows.
#pragma once

#include <type_traits>

#include "ge_device.h"

namespace ge {

// acc[fn][fm]: the swapped-operand accumulators of the tile kernels (lane half
// h of row r32 holds columns 8G + 4h + e in element 4G + e); mw, nw: the wave
// tile's first row and column; m0, bm: the workgroup tile's rows.
template <int KIND, int DOUT, int FM, int FN>
__device__ __forceinline__ void res_epilogue_kind(const KernelArgs& p, const ResArgs& q, const f32x16 (&acc)[FN][FM],
                                                  int mw, int nw, int lane) {
    const int r32 = lane & 31, h = lane >> 5;
    const int M = p.m, N = p.n;
    constexpr bool mask = KIND == GE_EPILOG_RELU_AUX_BIAS, keep = KIND == GE_EPILOG_GELU_AUX_BIAS;
    const bool row_bias = p.axis == GE_BIAS_ROW;
    float s = 1.0f;
    if (p.scale_a) s *= *p.scale_a;
    if (p.scale_b) s *= *p.scale_b;
    float rs[FM], br[FM];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int m = min(mw + fm * 32 + r32, M - 1);   // rows past the edge are never stored
        rs[fm] = q.row_scale ? s * q.row_scale[m] : s;
        br[fm] = p.bias && row_bias ? load_scalar<DOUT>(p.bias, m) : 0.0f;
    }
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) {
        const int nb = nw + fn * 32;
        uint32_t bits[FM];
#pragma unroll
        for (int fm = 0; fm < FM; ++fm) bits[fm] = 0u;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int nc = nb + 16 * g + 8 * h;
            const bool full = nc + 8 <= N;
            float bc[8], cs[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bc[j] = 0.0f;
                cs[j] = 1.0f;
            }
            if (p.bias && !row_bias) {
                if (full) load8<DOUT>(p.bias, nc, bc);
                else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) bc[j] = nc + j < N ? load_scalar<DOUT>(p.bias, nc + j) : 0.0f;
                }
            }
            if (q.col_scale) {
                if (full) load8<GE_F32>(q.col_scale, nc, cs);
                else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) cs[j] = nc + j < N ? q.col_scale[nc + j] : 1.0f;
                }
            }
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) {
                const int m = mw + fm * 32 + r32;
                const bool mok = m < M;
                const f32x16 a = acc[fn][fm];
                float v[8], pre[8], r[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[8 * g + e]),
                                                               __float_as_uint(a[8 * g + 4 + e]), false, false);
                    v[e] = __uint_as_float(sw[0]);
                    v[4 + e] = __uint_as_float(sw[1]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = 0.0f;
                if (q.res && mok) {
                    const int64_t idx = (int64_t)m * q.ldr + nc;
                    if (full) load8<DOUT>(q.res, idx, r);
                    else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) r[j] = nc + j < N ? load_scalar<DOUT>(q.res, idx + j) : 0.0f;
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    pre[j] = v[j] * rs[fm] * cs[j] + (bc[j] + br[fm]);
                    if (mask && pre[j] > 0.0f && nc + j < N) bits[fm] |= 1u << (16 * g + 8 * h + j);
                    v[j] = activate(KIND, pre[j]) + r[j];
                }
                if (mok) {
                    const int64_t idx = (int64_t)m * p.ldd + nc;
                    if (full) store8<DOUT>(p.D, idx, v);
                    else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (nc + j < N) store_one<DOUT>(p.D, idx + j, v[j]);
                    }
                    if (keep) store_pre8<DOUT>(p, m, nc, pre);
                }
            }
        }
        if (mask) {
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) {
                const int m = mw + fm * 32 + r32;
                const uint32_t w = bits[fm] | (uint32_t)__shfl_xor((int)bits[fm], 32);
                if (h == 0 && m < M && (nb >> 5) < p.ldaux) p.aux[(int64_t)m * p.ldaux + (nb >> 5)] = w;
            }
        }
    }
}

template <int DOUT, int FM, int FN, int BN, int NT>
__device__ __forceinline__ void res_epilogue(const KernelArgs& p, const ResArgs& q, const f32x16 (&acc)[FN][FM], int m0,
                                             int bm, int mw, int nw, int tn, int lane, int tid) {
    switch (p.epilog) {
    case GE_EPILOG_RELU_BIAS: res_epilogue_kind<GE_EPILOG_RELU_BIAS, DOUT, FM, FN>(p, q, acc, mw, nw, lane); break;
    case GE_EPILOG_RELU_AUX_BIAS: res_epilogue_kind<GE_EPILOG_RELU_AUX_BIAS, DOUT, FM, FN>(p, q, acc, mw, nw, lane); break;
    case GE_EPILOG_GELU_BIAS: res_epilogue_kind<GE_EPILOG_GELU_BIAS, DOUT, FM, FN>(p, q, acc, mw, nw, lane); break;
    case GE_EPILOG_GELU_AUX_BIAS: res_epilogue_kind<GE_EPILOG_GELU_AUX_BIAS, DOUT, FM, FN>(p, q, acc, mw, nw, lane); break;
    case GE_EPILOG_TANH_BIAS: res_epilogue_kind<GE_EPILOG_TANH_BIAS, DOUT, FM, FN>(p, q, acc, mw, nw, lane); break;
    default: res_epilogue_kind<GE_EPILOG_BIAS, DOUT, FM, FN>(p, q, acc, mw, nw, lane); break;   // NONE: no bias pointer
    }
    // mask words of the row padding that no tile covers
    if (p.epilog == GE_EPILOG_RELU_AUX_BIAS && tn == p.tiles_n - 1) {
        const int w0 = (p.tiles_n * BN) >> 5, nw = p.ldaux - w0;
        if (nw > 0) {
            for (int idx = tid; idx < bm * nw; idx += NT) {
                const int row = m0 + idx / nw;
                if (row < p.m) p.aux[(int64_t)row * p.ldaux + w0 + idx % nw] = 0u;
            }
        }
    }
}

}  // namespace ge
