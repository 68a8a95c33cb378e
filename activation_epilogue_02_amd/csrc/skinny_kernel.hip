// skinny_kernel.hip -- the residual product for few rows (m <= 64) and a
// weight given n x k, in 16-bit, E4M3 and block-scaled types.
//
// With so few rows every weight element is used at most 64 times, so the
// kernel is bound by streaming W once.  One workgroup takes 16 * RG columns of
// D (rows of W) and all of K; its eight waves split K in spans of 128 bytes of
// a row and their sums meet in LDS in wave order, so no partial sum leaves
// the CU and the call is one launch without a workspace: an exchange between
// workgroups costs 4 us and the partials' traffic (res_split in api.cpp), as
// long as 20 MB of W take to stream and more.
//  * A load instruction takes whole 128-byte lines (lane l: row l / 8, chunk
//    l % 8): fetched in the operand layout (lane: row l % 16, chunk l / 16) an
//    instruction touches 16 half lines, and the 16 x 4096 x 16384 bf16 product
//    took 43 us.  Each wave turns a span to the operand layout through 2 KB of LDS
//    per 16 rows of its own (no barrier), chunks XOR-swizzled by row / 2, so that
//    neither side meets a bank conflict: lane (r = lane % 16, q = lane / 16)
//    reads chunks q and 4 + q of row r, which are its K values in the 16x16x32
//    instruction (two of them per span) and in the 16x16x128 one (one per
//    span; its four 32-value blocks are the chunk pairs, so lane q's block
//    scale is byte q of the row's scale word).
//  * U spans are in flight in registers at all times: a span's slot is
//    loaded again as soon as its bytes are in LDS.
//  * x (m rows, read by every workgroup from L2) takes the same path.
//  * Workgroups start at different spans of their waves' K ranges: the rows of
//    W are often a power of two apart, and in lock-step all of them would ask the
//    same few memory channels.
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
    constexpr int TILES = RG + MB;   // 16-row groups of W, then of x
    constexpr int STAGE = kWaves * TILES * 2048, RED = kWaves * NB * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t smem[STAGE > RED ? STAGE : RED];
    f32x4(*red)[NB][64] = (f32x4(*)[NB][64])smem;   // the waves' sums, after the K loop
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
    auto row_of = [&](int tile, int row) __attribute__((always_inline)) {
        if (tile < RG) return (const uint8_t*)p.B + (int64_t)min(n0 + 16 * tile + row, N - 1) * p.ldb * ESZ;
        return (const uint8_t*)p.A + (int64_t)min(16 * (tile - RG) + row, M - 1) * p.lda * ESZ;
    };
    auto scales_of = [&](int tile) __attribute__((always_inline)) {
        if (tile < RG) return a.sb + (int64_t)min(n0 + 16 * tile + r, N - 1) * a.ld;
        return a.sa + (int64_t)min(16 * (tile - RG) + r, M - 1) * a.ld;
    };
    const uint8_t* src[TILES][2];   // this lane's rows of the loads
    const uint8_t* sc[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        src[i][0] = row_of(i, lane >> 3) + 16 * (lane & 7);
        src[i][1] = row_of(i, 8 + (lane >> 3)) + 16 * (lane & 7);
        sc[i] = MX ? scales_of(i) : nullptr;
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

    // spans in flight: what 256 registers per lane hold beside the rest
    constexpr int U = MX ? (TILES <= 2 ? 4 : TILES <= 4 ? 2 : 1) : TILES <= 2 ? 8 : TILES <= 3 ? 6 : TILES <= 4 ? 4 : TILES <= 5 ? 3 : 2;
    struct Slot {
        u32x4 v[TILES][2];
        uint32_t sc[TILES];
    };
    uint8_t* st = smem + wave * (TILES * 2048);
    const int put0 = (lane >> 3) * 128 + (((lane & 7) ^ ((lane >> 4) & 7)) << 4);         // row lane / 8
    const int put1 = (8 + (lane >> 3)) * 128 + (((lane & 7) ^ (4 + (lane >> 4))) << 4);   // row 8 + lane / 8
    const int get0 = r * 128 + ((q ^ (r >> 1)) << 4), get1 = r * 128 + (((4 + q) ^ (r >> 1)) << 4);
    const int count = s_full - s_begin;
    const int rot = count > 0 ? nblk % count : 0;
    auto load = [&](Slot& t, int i) __attribute__((always_inline)) {   // full span i of this wave
        int s = s_begin + i + rot;
        if (s >= s_full) s -= count;
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u32x4* g = (const u32x4*)(src[k][j] + (int64_t)s * 128);
                t.v[k][j] = k < RG ? __builtin_nontemporal_load(g) : *g;
            }
            if constexpr (MX) t.sc[k] = *(const uint32_t*)(sc[k] + 4 * s);
        }
    };
    // the slot's span through LDS, its next span's loads (where `more`), its MFMAs
    auto take = [&](Slot& t, int next, bool more) __attribute__((always_inline)) {
        uint32_t w[TILES];
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            *(u32x4*)(st + k * 2048 + put0) = t.v[k][0];
            *(u32x4*)(st + k * 2048 + put1) = t.v[k][1];
            w[k] = MX ? t.sc[k] >> (8 * q) : 0u;
        }
        // (a wave's LDS operations keep their order: only the compiler must not move them)
        asm volatile("" ::: "memory");
        if (more) load(t, next);
        u32x4 f[TILES][2];
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            f[k][0] = *(const u32x4*)(st + k * 2048 + get0);
            f[k][1] = *(const u32x4*)(st + k * 2048 + get1);
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int b = 0; b < MB; ++b)
                acc[g][b] = span_mfma<DIN>(f[g][0], f[g][1], f[RG + b][0], f[RG + b][1], w[g], w[RG + b], acc[g][b]);
    };
    // fewer spans than `most`: the missing ones are read as the last (a branch
    // around a load would make every wait one for all loads), and not used
    Slot t[U];
    auto few = [&](auto most) __attribute__((always_inline)) {
        constexpr int L = decltype(most)::value;
#pragma unroll
        for (int u = 0; u < L; ++u) load(t[u], min(u, count - 1));
#pragma unroll
        for (int u = 0; u < L; ++u)
            if (u < count) take(t[u], 0, false);
    };
    if (count >= U) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(t[u], u);
        int i = 0;
        for (; i + 2 * U <= count; i += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) take(t[u], i + U + u, true);
        }
        // at least U and fewer than 2 U are left
#pragma unroll
        for (int u = 0; u < U; ++u) take(t[u], i + U + u, i + U + u < count);
        i += U;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < count) take(t[u], 0, false);
    } else if (2 * count > U) {
        few(std::integral_constant<int, U>{});
    } else if (count > 0) {
        few(std::integral_constant<int, (U + 1) / 2>{});
    }
    if (full >= s_begin && full < s_end) {
        // the ragged last span: what lies beyond k is zero in both operands
        // (0 * NaN would not vanish), and its block scales are 1
        const int64_t off = (int64_t)full * 128 + 16 * q;
        const int blocks = MX ? a.kb - 4 * full : 0;   // valid scale bytes of the span's word
        uint32_t keep = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < blocks) keep |= 0xffu << (8 * j);
        u32x4 f[TILES][2];
        uint32_t w[TILES];
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            const uint8_t* row = row_of(k, r);
            f[k][0] = chunk_masked<ESZ>(row, off, bytes);
            f[k][1] = chunk_masked<ESZ>(row, off + 64, bytes);
            w[k] = MX ? ((*(const uint32_t*)(sc[k] + 4 * full) & keep) | (0x7f7f7f7fu & ~keep)) >> (8 * q) : 0u;
        }
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int b = 0; b < MB; ++b)
                acc[g][b] = span_mfma<DIN>(f[g][0], f[g][1], f[RG + b][0], f[RG + b][1], w[g], w[RG + b], acc[g][b]);
    }
    __syncthreads();   // `red` lies over the waves' stages
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
