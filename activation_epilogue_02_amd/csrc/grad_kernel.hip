// grad_kernel.hip -- the element-wise part of the residual product's backward
// pass: dP = dD * act'(aux), its transpose, and the bias gradient's partial
// sums, in one pass over dD and aux; and the plain transpose of an operand.
//
// A workgroup takes a 64 x 64 tile: 16-byte loads along the rows, the bias
// sums over the tile's rows (or columns) from the fp32 values, and the
// rounded tile through LDS for the transposed store, so both orders are
// written in whole lines.  Bound by memory.
#include "bias_sum.h"
#include "grad_params.h"

namespace ge {
namespace {

constexpr int TS = 64;   // tile rows and columns

// GELU' of a stored pre-activation.  One that left the type's range is stored as an
// infinity (fp16: beyond 65504), where the formula is inf * 0: beyond 30 GELU' is 1 or 0
// to the last bit of fp32, so the argument is cut there.  NaN stays NaN.
__device__ __forceinline__ float gelu_slope(float x) {
    x = x > 30.0f ? 30.0f : x;
    return gelu_tanh_deriv(x < -30.0f ? -30.0f : x);
}

template <int DT, int KIND>
__global__ void __launch_bounds__(256) grad_prepare(GradArgs p) {
    constexpr int E = 16 / Elem<DT>::size, CH = TS / E, RP = 256 / CH;   // rows per pass
    typedef typename Elem<DT>::T T;
    __shared__ T tile[TS][TS + E / 2 + 1];   // [column][row]
    __shared__ float sums[TS][RP + 1];       // COL: [column][row group]; ROW: [row][chunk]
    const int t = threadIdx.x, ch = t % CH, rg = t / CH;
    const int c0 = blockIdx.x * TS, r0 = blockIdx.y * TS;
    const int M = p.rows, N = p.cols;
    const bool row_axis = p.axis == GE_BIAS_ROW;
    const int n = c0 + ch * E;
    float col[E];
#pragma unroll
    for (int e = 0; e < E; ++e) col[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < TS / RP; ++i) {
        const int lr = rg + i * RP, m = r0 + lr;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.0f;
        T raw[E];
#pragma unroll
        for (int e = 0; e < E; ++e) raw[e] = (T)0;
        if (m < M && n < N) {
            const bool full = n + E <= N;
            const T* src = (const T*)p.src + (int64_t)m * p.ld + n;
            if (full) {
                const u32x4 w = *(const u32x4*)src;
                __builtin_memcpy(raw, &w, 16);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (n + e < N) raw[e] = src[e];
            }
            if constexpr (KIND != GRAD_COPY) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = load_scalar<DT>(raw, e);
            }
            if constexpr (KIND == GRAD_MASK) {
                // E columns of one mask word
                const uint32_t w = ((const uint32_t*)p.aux)[(int64_t)m * p.ldaux + (n >> 5)] >> (n & 31);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = (w >> e) & 1u ? v[e] : 0.0f;
            }
            if constexpr (KIND == GRAD_GELU) {
                const T* ax = (const T*)p.aux + (int64_t)m * p.ldaux + n;
                T pre[E];
                if (full) {
                    const u32x4 w = *(const u32x4*)ax;
                    __builtin_memcpy(pre, &w, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) pre[e] = n + e < N ? ax[e] : (T)0;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] *= gelu_slope(load_scalar<DT>(pre, e));
            }
            if constexpr (KIND == GRAD_MASK || KIND == GRAD_GELU) {
                // dP is rounded to the operands' type, half a step of each value: the products take it
                // in 16 bits.  In fp32 they would run on the fp32 matrix instruction, at a sixteenth
                // of the rate; as two 16-bit terms, at half.  The gradients' error, their own rounding
                // included, is 2^0.5 times as large for it (8192 x 4096 x 16384 bf16, GELU: 0.0024 of their
                // size against 0.0017); dbias below sums the unrounded values.
#pragma unroll
                for (int e = 0; e < E; ++e) store_one<DT>(raw, e, v[e]);
                if (p.dst) {
                    T* d = (T*)p.dst + (int64_t)m * p.ldd + n;
                    if (full) {
                        u32x4 w;
                        __builtin_memcpy(&w, raw, 16);
                        *(u32x4*)d = w;
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (n + e < N) d[e] = raw[e];
                    }
                }
            }
        }
        if constexpr (KIND != GRAD_COPY) {
            if (row_axis) {
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) s += v[e];
                sums[lr][ch] = s;
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) col[e] += v[e];
            }
        }
        if (p.dst_t) {
#pragma unroll
            for (int e = 0; e < E; ++e) tile[ch * E + e][lr] = raw[e];
        }
    }
    if constexpr (KIND != GRAD_COPY) {
        if (!row_axis) {
#pragma unroll
            for (int e = 0; e < E; ++e) sums[ch * E + e][rg] = col[e];
        }
    }
    __syncthreads();
    if constexpr (KIND != GRAD_COPY) {
        if (p.partial && t < TS) {
            float s = 0.0f;
            for (int i = 0; i < (row_axis ? CH : RP); ++i) s += sums[t][i];
            if (row_axis) {
                if (r0 + t < M) p.partial[(int64_t)blockIdx.x * M + r0 + t] = s;
            } else if (c0 + t < N) {
                p.partial[(int64_t)blockIdx.y * N + c0 + t] = s;
            }
        }
    }
    if (!p.dst_t) return;
#pragma unroll
    for (int i = 0; i < TS / RP; ++i) {
        const int lc = rg + i * RP, m = r0 + ch * E;   // column lc of the tile, its rows m .. m + E - 1
        if (c0 + lc >= N || m >= M) continue;
        T raw[E];
#pragma unroll
        for (int e = 0; e < E; ++e) raw[e] = tile[lc][ch * E + e];
        T* d = (T*)p.dst_t + (int64_t)(c0 + lc) * p.ldt + m;
        if (m + E <= M) {
            u32x4 w;
            __builtin_memcpy(&w, raw, 16);
            *(u32x4*)d = w;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (m + e < M) d[e] = raw[e];
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(256) grad_bias(const float* partial, int parts, int len, void* out) {
    __shared__ float red[kSumGroups][kSumCols + 1];
    sum_partials<DT>(partial, parts, len, out, blockIdx.x, threadIdx.x, red);
}

template <int DT>
void (*pick(int kind))(GradArgs) {
    switch (kind) {
    case GRAD_COPY: return grad_prepare<DT, GRAD_COPY>;
    case GRAD_PLAIN: return grad_prepare<DT, GRAD_PLAIN>;
    case GRAD_MASK: return grad_prepare<DT, GRAD_MASK>;
    case GRAD_GELU: return grad_prepare<DT, GRAD_GELU>;
    }
    return nullptr;
}

}  // namespace

int launch_grad_prepare(int type, int kind, const GradArgs& a, void* stream) {
    void (*fn)(GradArgs) = type == GE_F32 ? pick<GE_F32>(kind) : type == GE_F16 ? pick<GE_F16>(kind)
                           : type == GE_BF16 ? pick<GE_BF16>(kind) : nullptr;
    if (!fn) return (int)hipErrorInvalidDeviceFunction;
    const dim3 grid((unsigned)((a.cols + TS - 1) / TS), (unsigned)((a.rows + TS - 1) / TS));
    hipLaunchKernelGGL(fn, grid, dim3(256), 0, (hipStream_t)stream, a);
    return (int)hipGetLastError();
}

int launch_grad_bias(int type, const float* partial, int parts, int len, void* out, void* stream) {
    void (*fn)(const float*, int, int, void*) = type == GE_F32 ? grad_bias<GE_F32> : type == GE_F16 ? grad_bias<GE_F16>
                                                : type == GE_BF16 ? grad_bias<GE_BF16> : nullptr;
    if (!fn) return (int)hipErrorInvalidDeviceFunction;
    hipLaunchKernelGGL(fn, dim3((unsigned)((len - 1) / kSumCols + 1)), dim3(256), 0, (hipStream_t)stream, partial, parts,
                       len, out);
    return (int)hipGetLastError();
}

}  // namespace ge
