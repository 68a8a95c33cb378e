// skinny_kernel.hip -- the residual product for few rows (m <= 64) and a
// weight given n x k, in 16-bit, E4M3 and block-scaled types.
//
// With so few rows every weight element is used at most 64 times, so the
// kernel is bound by streaming W once.  One workgroup takes 16 * RG columns of
// D (rows of W) and all of K; its eight waves split K in spans of 128 bytes of
// a row and their sums meet in LDS in wave order, so no partial sum leaves
// the CU and the call is one launch without a workspace: an exchange between
// workgroups costs about 6 us, as long as 30 MB of W take to stream.
//  * W goes from memory to the matrix instruction's operand registers
//    directly: lane (r = lane % 16, q = lane / 16) takes the 16-byte chunks q
//    and 4 + q of row r's span, which are its K values in the 16x16x32
//    instruction (two of them per span) and in the 16x16x128 one (one per
//    span; its four 32-value blocks are the chunk pairs, so lane q's block
//    scale is byte q of the row's scale word).
//  * A wave's loads of U spans all go out before its first MFMA, so the
//    memory latency is paid once per batch.
//  * x (m rows, read by every workgroup from L2) takes the same pattern.
//  * The epilogue's operands (bias, scales, residual) are fetched before
//    the K loop, so that their latency hides under it.
#include <type_traits>

#include "ge_device.h"

namespace ge {
namespace {

constexpr int kWaves = 8;

// read in place of an absent bias or residual, or of an absent scale
__device__ const uint32_t kNoTerm[4] = {0u, 0u, 0u, 0u};
__device__ const float kNoScale[4] = {1.0f, 1.0f, 1.0f, 1.0f};

// the 16-byte chunk at byte `off` of a row of `bytes` bytes; what lies
// beyond reads as zero
template <int ESZ>
__device__ __forceinline__ u32x4 chunk_masked(const uint8_t* row, int64_t off, int64_t bytes) {
    u32x4 r = {0u, 0u, 0u, 0u};
    if (off + 16 <= bytes) return *(const u32x4*)(row + off);
    if (off >= bytes) return r;
    if constexpr (ESZ == 2) {
        uint16_t t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = off + 2 * e < bytes ? *(const uint16_t*)(row + off + 2 * e) : (uint16_t)0;
        __builtin_memcpy(&r, t, 16);
    } else {
        uint8_t t[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) t[e] = off + e < bytes ? row[off + e] : (uint8_t)0;
        __builtin_memcpy(&r, t, 16);
    }
    return r;
}

template <int DIN>
__device__ __forceinline__ f32x4 span_mfma(u32x4 w0, u32x4 w1, u32x4 x0, u32x4 x1, uint32_t sw, uint32_t sx, f32x4 c) {
    if constexpr (DIN == GE_BF16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w0), __builtin_bit_cast(bf16x8, x0), c, 0,
                                                    0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w1), __builtin_bit_cast(bf16x8, x1), c,
                                                       0, 0, 0);
    } else if constexpr (DIN == GE_F16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w0), __builtin_bit_cast(f16x8, x0), c, 0, 0,
                                                   0);
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w1), __builtin_bit_cast(f16x8, x1), c, 0,
                                                      0, 0);
    } else {
        const i32x8 w = {(int)w0[0], (int)w0[1], (int)w0[2], (int)w0[3], (int)w1[0], (int)w1[1], (int)w1[2], (int)w1[3]};
        const i32x8 x = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        if constexpr (DIN == GE_MXF8_E4M3)
            return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, (int)sw, 0, (int)sx);
        else
            return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, 0, 0, 0);
    }
}

template <int DIN, int DOUT, int MB, int RG>
__global__ void __launch_bounds__(kWaves * 64) ge_skinny_kernel(KernelArgs p, ResArgs a) {
    constexpr bool MX = DIN == GE_MXF8_E4M3;
    constexpr int ESZ = DIN == GE_F16 || DIN == GE_BF16 ? 2 : 1;
    constexpr int NB = MB * RG;   // 16 x 16 blocks of D
    static_assert(NB <= kWaves, "one block per wave in the epilogue");
    __shared__ f32x4 red[kWaves][NB][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int nblk = blockIdx.x, n0 = nblk * 16 * RG;
    const int M = p.m, N = p.n;
    const int64_t bytes = (int64_t)p.k * ESZ;   // of a row
    const int spans = (int)((bytes + 127) / 128), full = (int)(bytes / 128);
    const int per_wave = (spans + kWaves - 1) / kWaves;
    // neighbouring workgroups start on different parts of x
    const int slot = (wave + nblk) % kWaves;
    const int s_begin = min(spans, slot * per_wave), s_end = min(spans, s_begin + per_wave);
    const int s_full = min(s_end, full);

    // rows beyond n (W) or m (x) feed outputs that are never stored: clamped
    const uint8_t* wrow[RG];
    const uint8_t* xrow[MB];
    const uint8_t* wsc[RG];
    const uint8_t* xsc[MB];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
        const int64_t n = min(n0 + 16 * g + r, N - 1);
        wrow[g] = (const uint8_t*)p.B + n * p.ldb * ESZ;
        wsc[g] = MX ? a.sb + n * a.ld : nullptr;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t m = min(16 * b + r, M - 1);
        xrow[b] = (const uint8_t*)p.A + m * p.lda * ESZ;
        xsc[b] = MX ? a.sa + m * a.ld : nullptr;
    }

    // this wave's block of the epilogue (the waves past NB repeat the last
    // one's loads) and its operands: lane (r, q) has row 16b + r, columns
    // n .. n + 3.  No branches: absent terms are read from the constants.
    const int blk = min(wave, NB - 1), eg = blk / MB, eb = blk % MB;
    const int em = 16 * eb + r, en = n0 + 16 * eg + 4 * q;
    typedef typename Elem<DOUT>::T T;
    typedef __attribute__((address_space(1))) const T GT;
    typedef __attribute__((address_space(1))) const float GF;
    const bool row_bias = p.axis == GE_BIAS_ROW;
    const int64_t mc = min(em, M - 1);
    GT* bias = p.bias ? (GT*)p.bias : (GT*)kNoTerm;
    GT* res = a.res ? (GT*)a.res : (GT*)kNoTerm;
    GF* cscale = a.col_scale ? (GF*)a.col_scale : (GF*)kNoScale;
    GF* rscale = a.row_scale ? (GF*)a.row_scale : (GF*)kNoScale;
    T braw[4], rraw[4];
    float cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = min(en + i, N - 1);
        braw[i] = bias[!p.bias ? 0 : row_bias ? (int)mc : n];
        rraw[i] = res[a.res ? mc * a.ldr + n : 0];
        cs[i] = cscale[a.col_scale ? n : 0];
    }
    const float rs = rscale[a.row_scale ? mc : 0];
    __builtin_amdgcn_sched_barrier(0);

    f32x4 acc[RG][MB];
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[g][b] = f32x4{0.f, 0.f, 0.f, 0.f};

    int s0 = s_begin;
    auto batch = [&](auto u_const) __attribute__((always_inline)) {
        constexpr int U = decltype(u_const)::value;
        u32x4 w0[U][RG], w1[U][RG], x0[U][MB], x1[U][MB];
        uint32_t sw[U][RG], sx[U][MB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t off = (int64_t)(s0 + u) * 128 + 16 * q;
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                w0[u][g] = __builtin_nontemporal_load((const u32x4*)(wrow[g] + off));
                w1[u][g] = __builtin_nontemporal_load((const u32x4*)(wrow[g] + off + 64));
                if constexpr (MX) sw[u][g] = *(const uint32_t*)(wsc[g] + 4 * (s0 + u));
            }
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                x0[u][b] = *(const u32x4*)(xrow[b] + off);
                x1[u][b] = *(const u32x4*)(xrow[b] + off + 64);
                if constexpr (MX) sx[u][b] = *(const uint32_t*)(xsc[b] + 4 * (s0 + u));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    acc[g][b] = span_mfma<DIN>(w0[u][g], w1[u][g], x0[u][b], x1[u][b], MX ? sw[u][g] >> (8 * q) : 0u,
                                               MX ? sx[u][b] >> (8 * q) : 0u, acc[g][b]);
            __builtin_amdgcn_sched_barrier(0);
        }
        s0 += U;
    };
    // spans per batch: about 128 registers of operands
    constexpr int U = MB + RG <= 2 ? 8 : MB + RG <= 4 ? 4 : 2;
    while (s0 + U <= s_full) batch(std::integral_constant<int, U>{});
    if constexpr (U > 4)
        if (s0 + 4 <= s_full) batch(std::integral_constant<int, 4>{});
    if constexpr (U > 2)
        if (s0 + 2 <= s_full) batch(std::integral_constant<int, 2>{});
    if (s0 < s_full) batch(std::integral_constant<int, 1>{});
    if (full >= s_begin && full < s_end) {
        // the ragged last span: what lies beyond k is zero in both operands
        // (0 * NaN would not vanish), and its block scales are 1
        const int64_t off = (int64_t)full * 128 + 16 * q;
        const int blocks = MX ? a.kb - 4 * full : 0;   // valid scale bytes of the span's word
        uint32_t keep = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < blocks) keep |= 0xffu << (8 * j);
        u32x4 w0[RG], w1[RG];
        uint32_t sw[RG];
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            w0[g] = chunk_masked<ESZ>(wrow[g], off, bytes);
            w1[g] = chunk_masked<ESZ>(wrow[g], off + 64, bytes);
            sw[g] = MX ? (*(const uint32_t*)(wsc[g] + 4 * full) & keep) | (0x7f7f7f7fu & ~keep) : 0u;
        }
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const u32x4 x0 = chunk_masked<ESZ>(xrow[b], off, bytes), x1 = chunk_masked<ESZ>(xrow[b], off + 64, bytes);
            const uint32_t sx = MX ? (*(const uint32_t*)(xsc[b] + 4 * full) & keep) | (0x7f7f7f7fu & ~keep) : 0u;
#pragma unroll
            for (int g = 0; g < RG; ++g)
                acc[g][b] = span_mfma<DIN>(w0[g], w1[g], x0, x1, sw[g] >> (8 * q), sx >> (8 * q), acc[g][b]);
        }
    }
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
        for (int b = 0; b < MB; ++b) red[wave][g * MB + b][lane] = acc[g][b];
    __syncthreads();
    if (wave >= NB) return;
    f32x4 sum = red[0][blk][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w][blk][lane];

    const int ep = p.epilog;
    float s = rs;
    if (p.scale_a) s *= *p.scale_a;
    if (p.scale_b) s *= *p.scale_b;
    const bool mok = em < M, mask = ep == GE_EPILOG_RELU_AUX_BIAS;
    float v[4], pre[4];
    uint32_t bits = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float bv, rv;
        if constexpr (DOUT == GE_F32) { bv = braw[i]; rv = rraw[i]; }
        else if constexpr (DOUT == GE_BF16) { bv = bf16_bits_to_f32(braw[i]); rv = bf16_bits_to_f32(rraw[i]); }
        else { bv = f16_bits_to_f32(braw[i]); rv = f16_bits_to_f32(rraw[i]); }
        pre[i] = sum[i] * s * cs[i] + bv;
        if (mask && pre[i] > 0.0f && en + i < N) bits |= 1u << (4 * q + i);
        v[i] = activate(ep, pre[i]) + rv;
    }
    auto store4 = [&](void* D, int64_t idx, const float* f) __attribute__((always_inline)) {
        if (en + 4 <= N) {
            if constexpr (DOUT == GE_F32) {
                *(f32x4*)((float*)D + idx) = f32x4{f[0], f[1], f[2], f[3]};
            } else {
                uint32_t w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (DOUT == GE_BF16)
                        w[i] = f32_to_bf16_bits(f[2 * i]) | ((uint32_t)f32_to_bf16_bits(f[2 * i + 1]) << 16);
                    else
                        w[i] = f32_to_f16_bits(f[2 * i]) | ((uint32_t)f32_to_f16_bits(f[2 * i + 1]) << 16);
                }
                *(u32x2*)((uint16_t*)D + idx) = u32x2{w[0], w[1]};
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (en + i < N) store_one<DOUT>(D, idx + i, f[i]);
        }
    };
    if (mok) {
        store4(p.D, (int64_t)em * p.ldd + en, v);
        if (ep == GE_EPILOG_GELU_AUX_BIAS) store4(p.aux, (int64_t)em * p.ldaux + en, pre);
    }
    if (mask) {
        // 16 columns a half-word; a row's padding is cleared by the last block
        uint16_t* row = (uint16_t*)p.aux + (int64_t)em * p.ldaux * 2;
        bits |= (uint32_t)__shfl_xor((int)bits, 16);
        bits |= (uint32_t)__shfl_xor((int)bits, 32);
        if (q == 0 && mok) {
            row[nblk * RG + eg] = (uint16_t)bits;
            if (nblk == p.tiles_n - 1 && eg == RG - 1)
                for (int hw = (nblk + 1) * RG; hw < p.ldaux * 2; ++hw) row[hw] = 0;
        }
    }
}

template <int DIN, int DOUT>
void (*pick(int mb, int rg))(KernelArgs, ResArgs) {
    if (rg == 1) return mb == 1 ? ge_skinny_kernel<DIN, DOUT, 1, 1> : mb == 2 ? ge_skinny_kernel<DIN, DOUT, 2, 1>
                                                                              : ge_skinny_kernel<DIN, DOUT, 4, 1>;
    return mb == 1 ? ge_skinny_kernel<DIN, DOUT, 1, 2> : mb == 2 ? ge_skinny_kernel<DIN, DOUT, 2, 2>
                                                                 : ge_skinny_kernel<DIN, DOUT, 4, 2>;
}

}  // namespace

int launch_skinny(int a_type, int d_type, int mb, int rg, const KernelArgs& args, const ResArgs& res, unsigned grid,
                  void* stream) {
    void (*fn)(KernelArgs, ResArgs) = nullptr;
    if (a_type == GE_F16 && d_type == GE_F16) fn = pick<GE_F16, GE_F16>(mb, rg);
    else if (a_type == GE_F16 && d_type == GE_F32) fn = pick<GE_F16, GE_F32>(mb, rg);
    else if (a_type == GE_BF16 && d_type == GE_BF16) fn = pick<GE_BF16, GE_BF16>(mb, rg);
    else if (a_type == GE_BF16 && d_type == GE_F32) fn = pick<GE_BF16, GE_F32>(mb, rg);
    else if (a_type == GE_F8_E4M3 && d_type == GE_BF16) fn = pick<GE_F8_E4M3, GE_BF16>(mb, rg);
    else if (a_type == GE_F8_E4M3 && d_type == GE_F16) fn = pick<GE_F8_E4M3, GE_F16>(mb, rg);
    else if (a_type == GE_F8_E4M3 && d_type == GE_F32) fn = pick<GE_F8_E4M3, GE_F32>(mb, rg);
    else if (a_type == GE_MXF8_E4M3 && d_type == GE_BF16) fn = pick<GE_MXF8_E4M3, GE_BF16>(mb, rg);
    else if (a_type == GE_MXF8_E4M3 && d_type == GE_F16) fn = pick<GE_MXF8_E4M3, GE_F16>(mb, rg);
    else if (a_type == GE_MXF8_E4M3 && d_type == GE_F32) fn = pick<GE_MXF8_E4M3, GE_F32>(mb, rg);
    if (!fn) return (int)hipErrorInvalidDeviceFunction;
    hipLaunchKernelGGL(fn, dim3(grid), dim3(kWaves * 64), 0, (hipStream_t)stream, args, res);
    return (int)hipGetLastError();
}

}  // namespace ge
