// res_epilogue.h -- the residual product's epilogue on a tile's fp32
// accumulators: D = R + act(s * row_scale[i] * col_scale[j] * C + bias), with
// the ReLU sign mask or the pre-activation as an optional second output.
//
// The residual is added after the activation, so a block's output leaves with
// the residual stream already in it and R is read where D is written, once.
// Each kind is compiled as a copy of its own, picked once per tile: one body
// that tests the kind per element is several times as much code, fetched cold
// at the end of every tile.
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

// acc[fn][fm]: the swapped-operand accumulators of the tile kernels (lane half
// h of row r32 holds columns 8G + 4h + e in element 4G + e); mw, nw: the wave
// tile's first row and column; m0, bm: the workgroup tile's rows.
//
// A lane's row is fetched and stored over all of the wave tile's columns before
// the next row: an instruction covers 32 bytes of each of 32 rows, and taken
// column group by column group the four quarters of a line are requested so
// far apart that the caches drop it in between.  The next row's residual goes
// out before this one is computed where the registers hold both (two rows a
// lane, 16-bit outputs); loaded where it is used, every load's latency is paid
// in turn.  terms: the column bias, then the column scales, of the workgroup
// tile's BN columns from n0 on, in LDS (in registers they spilled the 256 x 256
// tile).
template <int KIND, int DOUT, int FM, int FN, int BN>
__device__ __forceinline__ void res_epilogue_kind(const KernelArgs& p, const ResArgs& q, const f32x16 (&acc)[FN][FM],
                                                  int mw, int nw, int n0, int lane, int tid, int nt, float* terms) {
    const int r32 = lane & 31, h = lane >> 5;
    const int M = p.m, N = p.n;
    constexpr bool mask = KIND == GE_EPILOG_RELU_AUX_BIAS, keep = KIND == GE_EPILOG_GELU_AUX_BIAS;
    const bool row_bias = p.axis == GE_BIAS_ROW, col_bias = p.bias && !row_bias;
    const bool whole = nw + FN * 32 <= N;   // every column of the wave tile exists
    constexpr bool AHEAD = DOUT != GE_F32 && FM <= 2;
    constexpr int G = 2 * FN, RW = kRaw8<DOUT>;   // groups of 16 columns, 8 of a lane
    // groups a fetch takes: the row, or a line of an fp32 one
    constexpr int GB = DOUT == GE_F32 ? 2 : G;
    u32x4 res[AHEAD ? 2 : 1][GB][RW];
    auto fetch = [&](int fm, int g0, u32x4 (&t)[GB][RW]) __attribute__((always_inline)) {
        const int m = min(mw + fm * 32 + r32, M - 1);   // rows past the edge are never stored
#pragma unroll
        for (int g = 0; g < GB; ++g) {
            const int nc = nw + 16 * (g0 + g) + 8 * h;
            fetch8<DOUT>(q.res, (int64_t)m * q.ldr + nc, nc, N, whole, t[g]);
        }
    };
    if (q.res && GB == G) fetch(0, 0, res[0]);
    __syncthreads();   // every wave has read its last fragments
    for (int j = tid; j < BN; j += nt) {
        const bool in = n0 + j < N;
        terms[j] = col_bias && in ? load_scalar<DOUT>(p.bias, n0 + j) : 0.0f;
        terms[BN + j] = q.col_scale && in ? q.col_scale[n0 + j] : 1.0f;
    }
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
    __syncthreads();
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
        if (q.res && GB == G && (AHEAD ? fm + 1 < FM : fm > 0))
            fetch(AHEAD ? fm + 1 : fm, 0, res[AHEAD ? (fm + 1) & 1 : 0]);
        const int m = mw + fm * 32 + r32;
        const bool mok = m < M;
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
            const int nb = nw + fn * 32;
            if (q.res && GB < G) fetch(fm, 2 * fn, res[0]);
            uint32_t bits = 0u;
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
                const int g = 2 * fn + gg, nc = nb + 16 * gg + 8 * h;
                const f32x16 a = acc[fn][fm];
                const f32x4* tb = (const f32x4*)(terms + (nc - n0));
                const f32x4 b0 = tb[0], b1 = tb[1], c0 = tb[BN / 4], c1 = tb[BN / 4 + 1];
                float v[8], pre[8], r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = 0.0f;
                if (q.res) unpack8<DOUT>(res[AHEAD ? fm & 1 : 0][g % GB], r);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[8 * gg + e]),
                                                               __float_as_uint(a[8 * gg + 4 + e]), false, false);
                    v[e] = __uint_as_float(sw[0]);
                    v[4 + e] = __uint_as_float(sw[1]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float bc = j < 4 ? b0[j & 3] : b1[j & 3], cs = j < 4 ? c0[j & 3] : c1[j & 3];
                    pre[j] = v[j] * rs[fm] * cs + (bc + br[fm]);
                    if (mask && pre[j] > 0.0f && nc + j < N) bits |= 1u << (16 * gg + 8 * h + j);
                    v[j] = activate(KIND, pre[j]) + r[j];
                }
                if (mok) {
                    const int64_t idx = (int64_t)m * p.ldd + nc;
                    if (whole || nc + 8 <= N) store8<DOUT>(p.D, idx, v);
                    else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (nc + j < N) store_one<DOUT>(p.D, idx + j, v[j]);
                    }
                    if (keep) store_pre8<DOUT>(p, m, nc, pre);
                }
            }
            if (mask) {
                const uint32_t w = bits | (uint32_t)__shfl_xor((int)bits, 32);
                if (h == 0 && mok && (nb >> 5) < p.ldaux) p.aux[(int64_t)m * p.ldaux + (nb >> 5)] = w;
            }
        }
    }
}

// smem: the workgroup's LDS, at least 8 BN bytes, 16-byte aligned.
template <int DOUT, int FM, int FN, int BN, int NT>
__device__ __forceinline__ void res_epilogue(const KernelArgs& p, const ResArgs& q, const f32x16 (&acc)[FN][FM], int m0,
                                             int bm, int mw, int nw, int n0, int tn, int lane, int tid, void* smem) {
    auto run = [&](auto kind) __attribute__((always_inline)) {
        res_epilogue_kind<decltype(kind)::value, DOUT, FM, FN, BN>(p, q, acc, mw, nw, n0, lane, tid, NT, (float*)smem);
    };
    switch (p.epilog) {
    case GE_EPILOG_RELU_BIAS: run(std::integral_constant<int, GE_EPILOG_RELU_BIAS>{}); break;
    case GE_EPILOG_RELU_AUX_BIAS: run(std::integral_constant<int, GE_EPILOG_RELU_AUX_BIAS>{}); break;
    case GE_EPILOG_GELU_BIAS: run(std::integral_constant<int, GE_EPILOG_GELU_BIAS>{}); break;
    case GE_EPILOG_GELU_AUX_BIAS: run(std::integral_constant<int, GE_EPILOG_GELU_AUX_BIAS>{}); break;
    case GE_EPILOG_TANH_BIAS: run(std::integral_constant<int, GE_EPILOG_TANH_BIAS>{}); break;
    default: run(std::integral_constant<int, GE_EPILOG_BIAS>{}); break;   // NONE: no bias pointer
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
