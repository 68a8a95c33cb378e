// norm_kernel.hip -- root-mean-square norm with the residual's addition and
// 8-bit outputs, and its backward pass (see include/ge_rms_norm.h for the
// formulas).
//
// Both directions are bound by memory: a handful of flops per value read.  A
// row stays in registers between its two (E4M3_ROW: three) uses, so each
// value crosses HBM once.  A thread holds `V` 16-byte chunks of its row,
// chunk t + i * T of thread t (whole lines per wave and load); the table in
// norm_params.h lists the shapes, and rows longer than 4096 chunks go through
// the *_long kernels, which read a row once per use (the second and third
// time from the caches).
#include "ge_device.h"
#include "norm_params.h"

namespace ge {
namespace {

constexpr int kBwdThreads = 512;   // workgroup of the backward pass (1024 for the rows that take more)
template <int DT> constexpr int kEpc = 16 / Elem<DT>::size;   // values per 16-byte chunk

// The 16-byte chunk `raw` as fp32 values.
template <int DT>
__device__ __forceinline__ void unpack(u32x4 raw, float* v) {
    if constexpr (DT == GE_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(raw[e]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == GE_BF16) {
                v[2 * i] = bf16_bits_to_f32(raw[i] & 0xffffu);
                v[2 * i + 1] = bf16_bits_to_f32(raw[i] >> 16);
            } else {
                v[2 * i] = f16_bits_to_f32(raw[i] & 0xffffu);
                v[2 * i + 1] = f16_bits_to_f32(raw[i] >> 16);
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ u32x4 pack(const float* v) {
    if constexpr (DT == GE_F32)
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    else
        return pack8_16bit<DT>(v);
}

// Chunk c of a vector of `cols` values; values at or beyond cols read as 0
// and are not touched in memory.
template <int DT>
__device__ __forceinline__ u32x4 load_chunk(const void* p, int c, int cols) {
    constexpr int E = kEpc<DT>;
    typedef typename Elem<DT>::T T;
    const T* q = (const T*)p + (int64_t)c * E;
    if ((c + 1) * (int64_t)E <= cols) return *(const u32x4*)q;
    u32x4 r = {0u, 0u, 0u, 0u};
    T t[E];
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = (int64_t)c * E + e < cols ? q[e] : (T)0;
    __builtin_memcpy(&r, t, 16);
    return r;
}

template <int DT>
__device__ __forceinline__ void store_chunk(void* p, int c, int cols, const float* v) {
    constexpr int E = kEpc<DT>;
    const int64_t j = (int64_t)c * E;
    if (j + E <= cols) {
        *(u32x4*)((uint8_t*)p + j * Elem<DT>::size) = pack<DT>(v);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (j + e < cols) store_one<DT>(p, j + e, v[e]);
    }
}

// E4M3 codes of the E values of chunk c, by the hardware's conversion (nearest
// even, NaN stays NaN).  It turns magnitudes that round above 448 into NaN, so
// they are clamped first unless CLAMP is false: values under 464 round to 448.
template <int E, bool CLAMP>
__device__ __forceinline__ void store_codes(uint8_t* y, int c, int cols, float* v) {
    uint32_t w[E / 4];
    if constexpr (CLAMP) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = __builtin_fabsf(v[e]) > 448.0f ? __builtin_copysignf(448.0f, v[e]) : v[e];
    }
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
        w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], lo, true);
    }
    const int64_t j = (int64_t)c * E;
    if (j + E <= cols) {
        if constexpr (E == 8) *(u32x2*)(y + j) = u32x2{w[0], w[1]};
        else *(uint32_t*)(y + j) = w[0];
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (j + e < cols) y[j + e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
    }
}

// Maximum that leaves NaN out (b first: a NaN in a is replaced).
__device__ __forceinline__ float max_num(float a, float b) { return a > b ? a : b; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = max_num(__shfl_xor(v, o), v);
    return v;
}

// Sum (or maximum) over the T threads of a row.  T = 64: one wave, no
// barrier.  Otherwise one barrier; `slot` alternates between calls, so that a
// wave may write the next call's values while another still reads this one's.
template <int T, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*red)[16], int slot) {
    v = MAX ? wave_max(v) : wave_sum(v);
    if constexpr (T > 64) {
        const int tid = threadIdx.x % T;
        if ((tid & 63) == 0) red[slot][tid >> 6] = v;
        __syncthreads();
        v = red[slot][0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) v = MAX ? max_num(red[slot][w], v) : v + red[slot][w];
    }
    return v;
}

// The block scale byte of a 32-column block with largest magnitude a, and
// the factor 2^-e of its codes (exact).  a in [2^k, 2^(k+1)) gives e = k - 8
// (448 = 1.75 * 2^8 is E4M3's largest value), at least -127, which every
// magnitude below 2^-118 gets, subnormals with them: k is the exponent field.
__device__ __forceinline__ uint32_t mx_scale(float a, float* f) {
    *f = 1.0f;
    if (!(a > 0.0f) || !(a < __builtin_inff())) return 127u;
    const int s = max((int)(__float_as_uint(a) >> 23) - 8, 0);
    *f = __uint_as_float((uint32_t)(254 - s) << 23);
    return (uint32_t)s;
}

// The scale of a row with largest magnitude a.  It is kept in the normal
// range, so that its reciprocal is finite.
__device__ __forceinline__ float row_scale(float a) {
    return a > 0.0f ? __builtin_fmaxf(a / 448.0f, 0x1p-126f) : 1.0f;
}

// y / s, rounded once (2^-24): the codes are those of the quotient.  A product
// with 1 / s lands beside the quotient for about every fourth value, and codes
// of values next to a border between two of them then differ.  With both scaled
// so that s is in [1, 2), which is exact, q = y * inv is off by an ulp or two,
// its remainder y - q s is exact, and one step with it rounds correctly (checked
// against divisions for 4e7 values, at and next to borders too).  s = inf gives 0,
// and NaN for infinite y, as the division does.
struct RowQuotient {
    float pow2, s, inv;
};
__device__ __forceinline__ RowQuotient row_quotient(float s) {
    if (s == __builtin_inff()) return {0.0f, 1.0f, 1.0f};
    const float pow2 = __uint_as_float((254u - (__float_as_uint(s) >> 23)) << 23);   // s is normal and below 2^120
    return {pow2, s * pow2, 1.0f / (s * pow2)};
}
__device__ __forceinline__ float divide(float y, const RowQuotient& d) {
    y *= d.pow2;
    const float q = y * d.inv;
    return __builtin_fmaf(__builtin_fmaf(-q, d.s, y), d.inv, q);
}

// The squared sum's rstd.
__device__ __forceinline__ float rstd_of(float ss, const NormArgs& p) { return 1.0f / sqrtf(ss * p.inv_cols + p.eps); }

// A workgroup takes rows b, b + blocks, ... (T = 64: each of its four waves a
// row of its own).
template <int DT, int OUT, int T, int V>
__global__ void __launch_bounds__(T < 256 ? 256 : T) norm_fwd(NormArgs p) {
    constexpr int E = kEpc<DT>, ES = Elem<DT>::size;
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ float red[2][16];
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const int cols = p.cols, C = (cols + E - 1) / E;
    int slot = 0;   // E4M3_ROW: 0, its maxima take 1; the others alternate from row to row
    // (T >= 256: the trip count is the same in the whole workgroup)
    for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < p.rows; row += (int64_t)p.blocks * RPB) {
        const int64_t off = row * p.ld * ES;
        u32x4 xr[V], rr[V], gr[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * T;
            xr[i] = rr[i] = gr[i] = u32x4{0u, 0u, 0u, 0u};
            if (c < C) {
                xr[i] = load_chunk<DT>((const uint8_t*)p.x + off, c, cols);
                if (p.res) rr[i] = load_chunk<DT>((const uint8_t*)p.res + off, c, cols);
                gr[i] = load_chunk<DT>(p.gamma, c, cols);
            }
        }
        float v[V][E], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            unpack<DT>(xr[i], v[i]);
            if (p.res) {
                float r[E];
                unpack<DT>(rr[i], r);
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] += r[e];
                // h is the rounded sum, and the norm is h's
                const u32x4 h = pack<DT>(v[i]);
                unpack<DT>(h, v[i]);
                const int c = t + i * T;
                if (p.h && c < C) store_chunk<DT>((uint8_t*)p.h + off, c, cols, v[i]);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) ss += v[i][e] * v[i][e];
        }
        const float rstd = rstd_of(row_reduce<T, false>(ss, red, slot), p);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float g[E];
            unpack<DT>(gr[i], g);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[i][e] = v[i][e] * rstd * g[e];
                if (OUT == GE_NORM_E4M3_ROW) amax = max_num(__builtin_fabsf(v[i][e]), amax);
            }
        }
        if constexpr (OUT == GE_NORM_PLAIN) {
            uint8_t* y = (uint8_t*)p.y + row * p.ldy * ES;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (t + i * T < C) store_chunk<DT>(y, t + i * T, cols, v[i]);
            slot ^= 1;
        } else if constexpr (OUT == GE_NORM_E4M3_ROW) {
            amax = row_reduce<T, true>(amax, red, 1);
            const float s = row_scale(amax);
            const RowQuotient d = row_quotient(s);
            if (t == 0) ((float*)p.scales)[row] = s;
            uint8_t* y = (uint8_t*)p.y + row * p.ldy;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] = divide(v[i][e], d);
                if (t + i * T < C) store_codes<E, false>(y, t + i * T, cols, v[i]);
            }
        } else {
            uint8_t* y = (uint8_t*)p.y + row * p.ldy;
            uint8_t* sc = (uint8_t*)p.scales + row * p.lds;
            // a 32-column block is 32 / E neighbouring lanes (T and the wave are
            // multiples of that)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = t + i * T;
                float a = 0.0f, f;
#pragma unroll
                for (int e = 0; e < E; ++e) a = max_num(__builtin_fabsf(v[i][e]), a);
#pragma unroll
                for (int o = 1; o < 32 / E; o <<= 1) a = max_num(__shfl_xor(a, o), a);
                const uint32_t byte = mx_scale(a, &f);
                if (c < C) {
#pragma unroll
                    for (int e = 0; e < E; ++e) v[i][e] *= f;
                    store_codes<E, true>(y, c, cols, v[i]);
                    if (c % (32 / E) == 0) sc[c / (32 / E)] = (uint8_t)byte;
                }
            }
            slot ^= 1;
        }
    }
}

// Rows of any length: one workgroup per row at a time, the row read again for each use.
template <int DT, int OUT>
__global__ void __launch_bounds__(1024) norm_fwd_long(NormArgs p) {
    constexpr int E = kEpc<DT>, ES = Elem<DT>::size, T = 1024;
    __shared__ float red[2][16];
    const int t = threadIdx.x;
    const int cols = p.cols, C = (cols - 1) / E + 1;
    for (int64_t row = blockIdx.x; row < p.rows; row += p.blocks) {
        const int64_t off = row * p.ld * ES;
        // h of chunk c: x + r rounded (first use), h itself once it is stored
        auto h_of = [&](int c, bool stored, float* v) __attribute__((always_inline)) {
            if (stored && p.h) {
                unpack<DT>(load_chunk<DT>((const uint8_t*)p.h + off, c, cols), v);
                return;
            }
            unpack<DT>(load_chunk<DT>((const uint8_t*)p.x + off, c, cols), v);
            if (p.res) {
                float r[E];
                unpack<DT>(load_chunk<DT>((const uint8_t*)p.res + off, c, cols), r);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] += r[e];
                const u32x4 h = pack<DT>(v);
                unpack<DT>(h, v);
                if (!stored && p.h) store_chunk<DT>((uint8_t*)p.h + off, c, cols, v);
            }
        };
        float ss = 0.0f;
        for (int64_t c = t; c < C; c += T) {
            float v[E];
            h_of((int)c, false, v);
#pragma unroll
            for (int e = 0; e < E; ++e) ss += v[e] * v[e];
        }
        const float rstd = rstd_of(row_reduce<T, false>(ss, red, 0), p);
        if (p.rstd && t == 0) p.rstd[row] = rstd;
        auto y_of = [&](int c, float* v) __attribute__((always_inline)) {
            float g[E];
            h_of(c, true, v);
            unpack<DT>(load_chunk<DT>(p.gamma, c, cols), g);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = v[e] * rstd * g[e];
        };
        float s = 1.0f;
        if constexpr (OUT == GE_NORM_E4M3_ROW) {
            float amax = 0.0f;
            for (int64_t c = t; c < C; c += T) {
                float v[E];
                y_of((int)c, v);
#pragma unroll
                for (int e = 0; e < E; ++e) amax = max_num(__builtin_fabsf(v[e]), amax);
            }
            amax = row_reduce<T, true>(amax, red, 1);
            s = row_scale(amax);
            if (t == 0) ((float*)p.scales)[row] = s;
        }
        [[maybe_unused]] const RowQuotient d = row_quotient(s);
        // every lane of a block's group takes part in its exchange, so the loop
        // runs to the same count in all of them
        for (int64_t c0 = 0; c0 < C; c0 += T) {
            const int64_t cl = c0 + t;
            const bool in = cl < C;
            const int c = in ? (int)cl : 0;
            float v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = 0.0f;
            if (in) y_of(c, v);
            if constexpr (OUT == GE_NORM_PLAIN) {
                if (in) store_chunk<DT>((uint8_t*)p.y + row * p.ldy * ES, c, cols, v);
            } else if constexpr (OUT == GE_NORM_E4M3_ROW) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = divide(v[e], d);
                if (in) store_codes<E, false>((uint8_t*)p.y + row * p.ldy, c, cols, v);
            } else {
                float a = 0.0f, f;
#pragma unroll
                for (int e = 0; e < E; ++e) a = max_num(__builtin_fabsf(v[e]), a);
#pragma unroll
                for (int o = 1; o < 32 / E; o <<= 1) a = max_num(__shfl_xor(a, o), a);
                const uint32_t byte = mx_scale(a, &f);
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] *= f;
                if (in) {
                    store_codes<E, true>((uint8_t*)p.y + row * p.ldy, c, cols, v);
                    if (c % (32 / E) == 0) ((uint8_t*)p.scales)[row * p.lds + c / (32 / E)] = (uint8_t)byte;
                }
            }
        }
        __syncthreads();   // before the next row's sums take red[0]
    }
}

// Backward: a workgroup of BT threads is RPB groups of T, each with a row of
// its own; group g of workgroup b takes rows g * blocks + b, then every
// blocks * RPB-th.  Its share of dgamma, a sum over rows, stays in registers;
// the groups' shares meet in LDS at the end, in group order, and are written
// once, to partial[b].  One workgroup per CU: every further one costs a row of
// partial sums to write and to read again.  512 threads, so that two rows fit
// into the registers (16384 x 4096 bf16 with the dgamma sum: 104 us at 512
// threads and 256 workgroups, 110 at 512 workgroups, 140 at 1024 threads,
// which spill, 128 and 106 at 256 threads and 256 and 512 workgroups).
template <int DT, int T, int V, int BT = (T > kBwdThreads ? T : kBwdThreads)>
__global__ void __launch_bounds__(BT) norm_bwd(NormArgs p) {
    constexpr int E = kEpc<DT>, ES = Elem<DT>::size;
    constexpr int RPB = BT / T;
    // the next row's loads go out before this row's reduction, where the
    // registers hold both rows
    constexpr bool AHEAD = V <= 2 && T <= kBwdThreads;
    __shared__ float red[RPB][2][16];
    __shared__ f32x4 comb[RPB > 1 ? RPB - 1 : 1][RPB > 1 ? V * E / 4 : 1][T];
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const int cols = p.cols, C = (cols + E - 1) / E;
    float acc[V][E];
    u32x4 gr[V], hr[V], dyr[V], dhr[V];
    float rstd_row = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        gr[i] = u32x4{0u, 0u, 0u, 0u};
        if (t + i * T < C) gr[i] = load_chunk<DT>(p.gamma, t + i * T, cols);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] = 0.0f;
    }
    auto load_row = [&](int64_t row) __attribute__((always_inline)) {
        const int64_t off = row * p.ld * ES;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * T;
            hr[i] = dyr[i] = dhr[i] = u32x4{0u, 0u, 0u, 0u};
            if (c < C && row < p.rows) {
                hr[i] = load_chunk<DT>((const uint8_t*)p.x + off, c, cols);
                dyr[i] = load_chunk<DT>((const uint8_t*)p.dy + off, c, cols);
                if (p.dh) dhr[i] = load_chunk<DT>((const uint8_t*)p.dh + off, c, cols);
            }
        }
        rstd_row = row < p.rows ? p.rstd[row] : 0.0f;
    };
    const int64_t stride = (int64_t)p.blocks * RPB;
    int slot = 0;
    if (AHEAD) load_row((int64_t)sub * p.blocks + blockIdx.x);
    // (the trip count is the same in the whole workgroup: group 0 has the
    // most rows, and a group past its last adds zeros)
    for (int64_t r0 = blockIdx.x; r0 < p.rows; r0 += stride) {
        const int64_t row = r0 + (int64_t)sub * p.blocks;
        const int64_t off = row * p.ld * ES;
        if (!AHEAD) load_row(row);
        u32x4 hc[V], dyc[V], dhc[V];
        const float rstd = rstd_row;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            hc[i] = hr[i];
            dyc[i] = dyr[i];
            dhc[i] = dhr[i];
            float h[E], dy[E], g[E];
            unpack<DT>(hc[i], h);
            unpack<DT>(dyc[i], dy);
            unpack<DT>(gr[i], g);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float n = h[e] * rstd;
                s += dy[e] * g[e] * n;
                acc[i][e] += dy[e] * n;
            }
        }
        if (AHEAD) load_row(row + stride);
        const float mean = row_reduce<T, false>(s, red[sub], slot) * p.inv_cols;
        slot ^= 1;
        // keep the packed values across the reduction, not the unpacked ones
#pragma unroll
        for (int i = 0; i < V; ++i) {
            asm volatile("" : "+v"(hc[i]), "+v"(dyc[i]), "+v"(dhc[i]));
            asm volatile("" : "+v"(gr[i]));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = t + i * T;
            float h[E], dy[E], g[E], dh[E], d[E];
            unpack<DT>(hc[i], h);
            unpack<DT>(dyc[i], dy);
            unpack<DT>(gr[i], g);
            unpack<DT>(dhc[i], dh);
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = rstd * (dy[e] * g[e] - h[e] * rstd * mean) + dh[e];
            if (c < C && row < p.rows) store_chunk<DT>((uint8_t*)p.dx + off, c, cols, d);
        }
    }
    if (!p.partial) return;
    if constexpr (RPB > 1) {
        if (sub > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int w = 0; w < E / 4; ++w)
                    comb[sub - 1][i * (E / 4) + w][t] =
                        f32x4{acc[i][4 * w], acc[i][4 * w + 1], acc[i][4 * w + 2], acc[i][4 * w + 3]};
        }
        __syncthreads();
        if (sub > 0) return;
        for (int g = 0; g < RPB - 1; ++g)
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int w = 0; w < E / 4; ++w) {
                    const f32x4 o = comb[g][i * (E / 4) + w][t];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][4 * w + e] += o[e];
                }
    }
    float* out = p.partial + (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t j = (int64_t)(t + i * T) * E;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (j + e < cols) out[j + e] = acc[i][e];
    }
}

// Rows of any length; the workgroup's dgamma sums live in its own row of
// `partial` (each value read and written by one thread only).
template <int DT>
__global__ void __launch_bounds__(1024) norm_bwd_long(NormArgs p) {
    constexpr int E = kEpc<DT>, ES = Elem<DT>::size, T = 1024;
    __shared__ float red[2][16];
    const int t = threadIdx.x, cols = p.cols, C = (cols - 1) / E + 1;
    int slot = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += p.blocks) {
        const int64_t off = row * p.ld * ES;
        const float rstd = p.rstd[row];
        float s = 0.0f;
        for (int64_t c = t; c < C; c += T) {
            float h[E], dy[E], g[E];
            unpack<DT>(load_chunk<DT>((const uint8_t*)p.x + off, (int)c, cols), h);
            unpack<DT>(load_chunk<DT>((const uint8_t*)p.dy + off, (int)c, cols), dy);
            unpack<DT>(load_chunk<DT>(p.gamma, (int)c, cols), g);
#pragma unroll
            for (int e = 0; e < E; ++e) s += dy[e] * g[e] * (h[e] * rstd);
        }
        const float mean = row_reduce<T, false>(s, red, slot) * p.inv_cols;
        slot ^= 1;
        for (int64_t c = t; c < C; c += T) {
            float h[E], dy[E], g[E], dh[E], d[E];
            unpack<DT>(load_chunk<DT>((const uint8_t*)p.x + off, (int)c, cols), h);
            unpack<DT>(load_chunk<DT>((const uint8_t*)p.dy + off, (int)c, cols), dy);
            unpack<DT>(load_chunk<DT>(p.gamma, (int)c, cols), g);
#pragma unroll
            for (int e = 0; e < E; ++e) dh[e] = 0.0f;
            if (p.dh) unpack<DT>(load_chunk<DT>((const uint8_t*)p.dh + off, (int)c, cols), dh);
            if (p.partial) {
                float* out = p.partial + (int64_t)blockIdx.x * cols + c * E;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (c * E + e < cols)
                        out[e] = (row == (int64_t)blockIdx.x ? 0.0f : out[e]) + dy[e] * (h[e] * rstd);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = rstd * (dy[e] * g[e] - h[e] * rstd * mean) + dh[e];
            store_chunk<DT>((uint8_t*)p.dx + off, (int)c, cols, d);
        }
    }
}

// dgamma[j] = sum over blocks b of partial[b][j], in a fixed order: a
// workgroup takes 32 columns, 32 groups of lanes every 32nd block each, then
// the groups in order.
template <int DT>
__global__ void __launch_bounds__(1024) norm_dgamma(NormArgs p) {
    __shared__ float red[32][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t j = (int64_t)blockIdx.x * 32 + c;
    float v = 0.0f;
    if (j < p.cols) {
#pragma unroll 4
        for (int b = g; b < p.blocks; b += 32) v += p.partial[(int64_t)b * p.cols + j];
    }
    red[g][c] = v;
    __syncthreads();
    if (g == 0 && j < p.cols) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][c];
        store_one<DT>(p.dgamma, j, s);
    }
}

typedef void (*NormFn)(NormArgs);

template <int DT, int OUT>
NormFn pick_fwd(NormShape s) {
    if (s.threads == 64) return s.chunks == 1 ? norm_fwd<DT, OUT, 64, 1> : norm_fwd<DT, OUT, 64, 2>;
    if (s.threads == 256)
        return s.chunks == 1 ? norm_fwd<DT, OUT, 256, 1>
               : s.chunks == 2 ? norm_fwd<DT, OUT, 256, 2>
               : s.chunks == 3 ? norm_fwd<DT, OUT, 256, 3> : norm_fwd<DT, OUT, 256, 4>;
    return s.chunks == 2 ? norm_fwd<DT, OUT, 1024, 2>
           : s.chunks == 4 ? norm_fwd<DT, OUT, 1024, 4> : norm_fwd_long<DT, OUT>;
}

template <int DT>
NormFn pick_fwd_out(int out, NormShape s) {
    return out == GE_NORM_PLAIN ? pick_fwd<DT, GE_NORM_PLAIN>(s)
           : out == GE_NORM_E4M3_ROW ? pick_fwd<DT, GE_NORM_E4M3_ROW>(s) : pick_fwd<DT, GE_NORM_MX>(s);
}

template <int DT>
NormFn pick_bwd(NormShape s) {
    if (s.threads == 64) return s.chunks == 1 ? norm_bwd<DT, 64, 1> : norm_bwd<DT, 64, 2>;
    if (s.threads == 256)
        return s.chunks == 1 ? norm_bwd<DT, 256, 1>
               : s.chunks == 2 ? norm_bwd<DT, 256, 2> : norm_bwd<DT, 256, 3>;
    if (s.threads == 512) return s.chunks == 2 ? norm_bwd<DT, 512, 2> : norm_bwd<DT, 512, 3>;
    return s.chunks == 2 ? norm_bwd<DT, 1024, 2>
           : s.chunks == 4 ? norm_bwd<DT, 1024, 4> : norm_bwd_long<DT>;
}

}  // namespace

int launch_norm_forward(int type, int out, NormShape s, const NormArgs& a, void* stream) {
    const NormFn fn = type == GE_F32 ? pick_fwd_out<GE_F32>(out, s)
                      : type == GE_F16 ? pick_fwd_out<GE_F16>(out, s) : pick_fwd_out<GE_BF16>(out, s);
    hipLaunchKernelGGL(fn, dim3((unsigned)a.blocks), dim3(s.threads < 256 ? 256u : (unsigned)s.threads), 0,
                       (hipStream_t)stream, a);
    return (int)hipGetLastError();
}

int launch_norm_backward(int type, NormShape s, const NormArgs& a, void* stream) {
    const NormFn fn = type == GE_F32 ? pick_bwd<GE_F32>(s)
                      : type == GE_F16 ? pick_bwd<GE_F16>(s) : pick_bwd<GE_BF16>(s);
    hipLaunchKernelGGL(fn, dim3((unsigned)a.blocks), dim3(s.threads > kBwdThreads ? s.threads : kBwdThreads), 0, (hipStream_t)stream, a);
    return (int)hipGetLastError();
}

int launch_norm_dgamma(int type, const NormArgs& a, void* stream) {
    const NormFn fn = type == GE_F32 ? norm_dgamma<GE_F32> : type == GE_F16 ? norm_dgamma<GE_F16> : norm_dgamma<GE_BF16>;
    hipLaunchKernelGGL(fn, dim3((unsigned)((a.cols - 1) / 32 + 1)), dim3(1024), 0, (hipStream_t)stream, a);
    return (int)hipGetLastError();
}

}  // namespace ge
