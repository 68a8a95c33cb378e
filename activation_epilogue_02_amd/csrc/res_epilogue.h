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

// Values of type DOUT, eight a lane, as loaded.
template <int DOUT> constexpr int kRaw8 = DOUT == GE_F32 ? 2 : 1;   // 16-byte words

template <int DOUT>
__device__ __forceinline__ void unpack8(const u32x4* w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DOUT == GE_F32) {
            v[i] = __uint_as_float(w[0][i]);
            v[4 + i] = __uint_as_float(w[1][i]);
        } else if constexpr (DOUT == GE_BF16) {
            v[2 * i] = bf16_bits_to_f32(w[0][i] & 0xffffu);
            v[2 * i + 1] = bf16_bits_to_f32(w[0][i] >> 16);
        } else {
            v[2 * i] = f16_bits_to_f32(w[0][i] & 0xffffu);
            v[2 * i + 1] = f16_bits_to_f32(w[0][i] >> 16);
        }
    }
}

// The eight values at element idx, of which those at columns nc + j < N exist
// (zeros for the rest); whole: all do, in every lane.
template <int DOUT>
__device__ __forceinline__ void fetch8(const void* p, int64_t idx, int nc, int N, bool whole, u32x4* w) {
    typedef typename Elem<DOUT>::T T;
    const T* q = (const T*)p + idx;
    if (whole || nc + 8 <= N) {
#pragma unroll
        for (int i = 0; i < kRaw8<DOUT>; ++i) w[i] = ((const u32x4*)q)[i];
    } else {
        T t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = nc + j < N ? q[j] : (T)0;
        __builtin_memcpy(w, t, sizeof t);
    }
}

// What 16 columns of the wave tile (8 of a lane) add: the residual of the
// lane's FM rows, and the column bias and scales.
template <int DOUT, int FM>
struct ResTerms {
    u32x4 res[FM][kRaw8<DOUT>];
    u32x4 bias[kRaw8<DOUT>];
    u32x4 scale[2];
};

// acc[fn][fm]: the swapped-operand accumulators of the tile kernels (lane half
// h of row r32 holds columns 8G + 4h + e in element 4G + e); mw, nw: the wave
// tile's first row and column; m0, bm: the workgroup tile's rows.
//
// The terms of 16 columns are fetched together, the next 16 columns' before
// these are computed where two sets fit the registers (two rows a lane, 16-bit
// outputs): loaded where they are used, each load's latency is paid in turn.
template <int KIND, int DOUT, int FM, int FN>
__device__ __forceinline__ void res_epilogue_kind(const KernelArgs& p, const ResArgs& q, const f32x16 (&acc)[FN][FM],
                                                  int mw, int nw, int lane) {
    const int r32 = lane & 31, h = lane >> 5;
    const int M = p.m, N = p.n;
    constexpr bool mask = KIND == GE_EPILOG_RELU_AUX_BIAS, keep = KIND == GE_EPILOG_GELU_AUX_BIAS;
    const bool row_bias = p.axis == GE_BIAS_ROW, col_bias = p.bias && !row_bias;
    const bool whole = nw + FN * 32 <= N;   // every column of the wave tile exists
    constexpr bool AHEAD = DOUT != GE_F32 && FM <= 2;
    ResTerms<DOUT, FM> terms[AHEAD ? 2 : 1];
    auto fetch = [&](int G, ResTerms<DOUT, FM>& t) __attribute__((always_inline)) {
        const int nc = nw + 16 * G + 8 * h;
        if (q.res) {
#pragma unroll
            for (int fm = 0; fm < FM; ++fm) {
                const int m = min(mw + fm * 32 + r32, M - 1);   // rows past the edge are never stored
                fetch8<DOUT>(q.res, (int64_t)m * q.ldr + nc, nc, N, whole, t.res[fm]);
            }
        }
        if (col_bias) fetch8<DOUT>(p.bias, nc, nc, N, whole, t.bias);
        if (q.col_scale) fetch8<GE_F32>(q.col_scale, nc, nc, N, whole, t.scale);
    };
    fetch(0, terms[0]);
    float s = 1.0f;
    if (p.scale_a) s *= *p.scale_a;
    if (p.scale_b) s *= *p.scale_b;
    float rs[FM], br[FM];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        const int m = min(mw + fm * 32 + r32, M - 1);
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
            const int G = 2 * fn + g;
            if (AHEAD ? G + 1 < 2 * FN : G > 0) fetch(AHEAD ? G + 1 : G, terms[AHEAD ? (G + 1) & 1 : 0]);
            const ResTerms<DOUT, FM>& t = terms[AHEAD ? G & 1 : 0];
            const int nc = nb + 16 * g + 8 * h;
            const bool full = whole || nc + 8 <= N;
            float bc[8], cs[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bc[j] = 0.0f;
                cs[j] = 1.0f;
            }
            if (col_bias) unpack8<DOUT>(t.bias, bc);
            if (q.col_scale) unpack8<GE_F32>(t.scale, cs);
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
                if (q.res) unpack8<DOUT>(t.res[fm], r);
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
