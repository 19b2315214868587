// Rows that become the next product's activations: RMS norm (with the
// residual's addition) and SwiGLU, each with a 16-bit or a quantised output.
//
//   norm:    h = x + r,  y = h (mean h^2 + eps)^-1/2 (w + offset)
//   SwiGLU:  y = silu(gate) up,  silu(g) = g / (1 + e^-g)
//   tokens:  s = max|y| / top over the row (top: E4M3 448, INT8 127; 1 for zeros, never 0), q = rnd(y / s)
//   blocks:  the same over 128 consecutive elements (E4M3)
//   MX:      E8M0 per 32: the exponent of max|y| less emax (E4M3 8, E2M1 2), q = rnd(y 2^(127 - e))
//
// All of it is bound by HBM: each element is read once and its code written
// once.  A row stays in registers, 8 consecutive elements a group, so the sum of
// squares, the maximum and the rounding need no second pass over memory; y is
// formed in fp32 from the unrounded h and rounded once.  Next to the bytes the
// instructions count (e^x, the quotients and the conversions of each element): SwiGLU
// of 16376 rows of 2048 in blocks with the library's e^x, divisions and a check of each
// code took 58 us, now 32 (5.3 TB/s); the norm of 8191 rows of 7168 with its residual,
// in tokens, 86 and now 76 (5.4 TB/s).  A call of few rows takes as long as its launch.
#include "hq_device.hpp"
#include "hq_layer.h"
#include "layer_rows.hpp"

namespace hq {

namespace {

struct RowParams {
    const void *x, *res, *w;
    void *sum, *out, *scale;
    int64_t rows, x_stride, res_stride, sum_stride;
    int width;
    float eps, w_offset;
    int silu, w_f32, fp4_or_i8;
};

enum class Quant { SAME16, TOKEN, BLOCK, MX };

__device__ __forceinline__ float amax8(const float (&y)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
    return m;
}

// Four E4M3 codes: rounded to nearest even, saturated at +-448, NaN kept (0x7F).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    auto sat = [](float v) { return fminf(fmaxf(v, -448.f), 448.f); };
    int pk = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
    pk = __builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), pk, true);
    uint32_t u = (uint32_t)pk;
    auto nan_fix = [&](int byte, float v) { u = v != v ? (u & ~(0xFFu << (8 * byte))) | (0x7Fu << (8 * byte)) : u; };
    nan_fix(0, a);
    nan_fix(1, b);
    nan_fix(2, c);
    nan_fix(3, d);
    return u;
}

// Four E4M3 codes of values that do not pass 464, the border to 480 (quotients of divide8, by a
// scale that takes the largest to 448): nothing to saturate, and a NaN comes as 0x7F or 0xFF, of
// which the sign is cleared (bytes whose low seven bits are all ones).
__device__ __forceinline__ uint32_t e4m3x4_below(float a, float b, float c, float d) {
    int pk = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    pk = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, pk, true);
    const uint32_t u = (uint32_t)pk;
    return u & ~(((u & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u);
}

// The scale that takes the largest value m to `top`; 1 for zeros.  Of a denormal m below some half
// `top` units of 2^-149 the quotient is 0, and zeros would be 0 / 0: one unit at least.
__device__ __forceinline__ float scale_of(float m, float top) { return m > 0.f ? fmaxf(m / top, 0x1p-149f) : 1.f; }

// v / s for eight values, s the scale that takes the largest to `top`.  With r = 1 / s after one
// Newton step, q0 = v r is within two units of v / s, and q0 - (q0 s - v) r within one half and
// the little that r is off by: the rounding to 8 bits sees no difference to a division but in a
// value within a unit of 2^-24 of a border.  Three instructions for each value in place of ten (SwiGLU,
// 16376 rows of 2048 in blocks: 32 us, with divisions 41; the norm of 8191 rows of 7168 in
// tokens: 76, 87).  Scales near the ends of the range, infinite
// ones and NaN take the division; a scale that is a denormal has lost bits, so the quotient is
// held at +-top there, NaN kept.
__device__ __forceinline__ void divide8(const float (&v)[8], float s, float top, float (&q)[8]) {
    if (s > 0x1p-90f && s < 0x1p90f) {
        float r = __builtin_amdgcn_rcpf(s);
        r = fmaf(fmaf(-s, r, 1.0f), r, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = v[i] * r;
            q[i] = fmaf(fmaf(q0, s, -v[i]), -r, q0);  // (with these signs a -0 stays one)
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = v[i] / s;
            q[i] = d > top ? top : d < -top ? -top : d;
        }
    }
}

// silu(g) = g / (1 + e^-g), as g / (1 + t) or g t / (1 + t) with t = e^-|g| <= 1 (no overflow at
// either end).  t = 2^(-|g| log2 e): the product's rounding, up to 2^-17 of t where |g| is
// large, is put back to first order.  |g| is held at 150, where t is 0 either way, so that an
// infinity has its limit or NaN as the formula has it.
__device__ __forceinline__ float silu(float g) {
    const float x = fmaxf(-fabsf(g), -150.f), h = x * 1.44269502f;
    const float rest = fmaf(x, 1.44269502f, -h) + x * 1.92596299e-8f;  // log2 e in two parts
    const float t0 = __builtin_amdgcn_exp2f(h), t = fmaf(t0, rest * 0.693147182f, t0);
    return (g >= 0.f ? g : g * t) * __builtin_amdgcn_rcpf(1.0f + t);
}
// ... and of g below kSiluFar (above -150), where the hardware's 2^h gives 0 for what would be a denormal
// t, while g t is a normal number down to some -92 (1 + t is 1): e^g = 2^f 2^n, 2^n behind the
// product.  A branch that no ordinary row takes; its test is one minimum for each value (8191 rows, us,
// without it: 2048 in tokens 22.3, now 21.2; MX 19.6, 20.5; with 2^f 2^n for all gates 24.7, 20.2).
constexpr float kSiluFar = -87.f;
__device__ __forceinline__ float silu_far(float g) {
    const float n = rintf(g * 1.44269502f);
    const float f = fmaf(g, 1.92596299e-8f, fmaf(g, 1.44269502f, -n));
    return ldexpf(g * __builtin_amdgcn_exp2f(f), (int)n);
}

// INT8 in -127..127, to nearest even; NaN becomes 0.
__device__ __forceinline__ uint32_t int8_code(float v) {
    return (uint32_t)(v != v ? 0 : (int)rintf(fminf(fmaxf(v, -127.f), 127.f))) & 0xFFu;
}

// E2M1 code of v with the sign of x: a midpoint of the grid 0, .5, 1, 1.5, 2, 3, 4, 6
// goes to the neighbour with the even mantissa bit.
__device__ __forceinline__ uint32_t e2m1_of(float x, float v) {
    const float a = fabsf(v);
    const uint32_t mag = (uint32_t)(a > 0.25f) + (uint32_t)(a >= 0.75f) + (uint32_t)(a > 1.25f) + (uint32_t)(a >= 1.75f) +
                         (uint32_t)(a > 2.5f) + (uint32_t)(a >= 3.5f) + (uint32_t)(a > 5.0f);
    return mag | ((__float_as_uint(x) >> 28) & 8u);
}

struct __attribute__((packed, aligned(1))) Any8 {
    uint2 v;
};

// Sum or maximum over the TPR threads of a row (TPR 64: one wave; else the whole workgroup).
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const float o = __shfl_xor(v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    if constexpr (TPR > 64) {
        constexpr int NW = TPR / 64;
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) v = MAX ? fmaxf(v, red[i]) : v + red[i];
    }
    return v;
}

// TPR threads hold a row of at most 8 NV TPR elements, thread i the groups of eight i, i + TPR,
// ..., so a block of 128 is 16 neighbouring lanes and one of 32 is 4.  VEC: width and strides
// are multiples of 8; without it no block scales.
template <bool BF16, Quant Q, int TPR, int NV, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void row_kernel(RowParams p) {
    static_assert(VEC || Q == Quant::SAME16 || Q == Quant::TOKEN, "block scales need whole groups");
    __shared__ float red[4][16];
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;  // rows per workgroup
    const int t = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
    if (RPW > 1 && row >= p.rows) return;  // (whole waves; no barrier below where RPW > 1)
    const int K = p.width;
    auto el = [&](int j) { return (j * TPR + t) * 8; };

    float y[NV][8];
    float ss = 0.f;
    if (p.silu) {
        const uint16_t* in = (const uint16_t*)p.x + row * p.x_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float g[8], u[8];
            unpack8<BF16>(load8<VEC>(in + el(j), K - el(j)), g);
            unpack8<BF16>(load8<VEC>(in + K + el(j), K - el(j)), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] = silu(g[i]) * u[i];
            float least = g[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) least = fminf(least, g[i]);
            if (__ballot(least < kSiluFar)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[j][i] = g[i] < kSiluFar && g[i] > -150.f ? silu_far(g[i]) * u[i] : y[j][i];
            }
        }
    } else {
        const uint16_t* x = (const uint16_t*)p.x + row * p.x_stride;
        const uint16_t* r = p.res ? (const uint16_t*)p.res + row * p.res_stride : nullptr;
        uint16_t* sum = p.sum ? (uint16_t*)p.sum + row * p.sum_stride : nullptr;
        v4u xv[NV], rv[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) xv[j] = load8<VEC>(x + el(j), K - el(j));
        if (r) {
#pragma unroll
            for (int j = 0; j < NV; ++j) rv[j] = load8<VEC>(r + el(j), K - el(j));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack8<BF16>(xv[j], y[j]);
            if (r) {
                float a[8];
                unpack8<BF16>(rv[j], a);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[j][i] += a[i];
            }
            if (sum) store8<VEC>(sum + el(j), pack8<BF16>(y[j]), K - el(j));
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += y[j][i] * y[j][i];
        }
        ss = row_reduce<TPR, false>(ss, red[0]);
        const float mean = ss / (float)K + p.eps;
        float rs = 1.0f / sqrtf(mean);
        // Squares at fp32's ends (sums of them that are denormals or 0 where eps does not cover it, or
        // infinite): the row is brought to 1..2 by a power of two first, eps with it in 64 bits.  (A NaN,
        // an infinity or a row of zeros has its rs already.)
        if (!(mean > 0x1p-100f && mean < INFINITY)) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) m = fmaxf(m, amax8(y[j]));
            m = row_reduce<TPR, true>(m, red[2]);
            if (m > 0.f && m < INFINITY && ss == ss) {
                const int e = ilogbf(m);
                float s2 = 0.f;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[j][i] = ldexpf(y[j][i], -e);
                        s2 += y[j][i] * y[j][i];
                    }
                s2 = row_reduce<TPR, false>(s2, red[3]);
                rs = (float)(1.0 / sqrt((double)s2 / K + ldexp((double)p.eps, -2 * e)));
            }
        }
        const uint16_t* w16 = (const uint16_t*)p.w;
        const float* w32 = (const float*)p.w;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float w[8];
            const int n = K - el(j);
            if (n <= 0) continue;  // zeros stay
            if (VEC || n >= 8) {
                if (p.w_f32) {
                    *(v4f*)&w[0] = *(const v4f*)(w32 + el(j));
                    *(v4f*)&w[4] = *(const v4f*)(w32 + el(j) + 4);
                } else {
                    unpack8<BF16>(ld16(w16 + el(j)), w);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = i >= n ? 0.f : p.w_f32 ? w32[el(j) + i] : bits16_to_f32<BF16>(w16[el(j) + i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (VEC || i < n) y[j][i] = y[j][i] * rs * (w[i] + p.w_offset);
        }
    }

    if constexpr (Q == Quant::SAME16) {
        uint16_t* out = (uint16_t*)p.out + row * K;
#pragma unroll
        for (int j = 0; j < NV; ++j) store8<VEC>(out + el(j), pack8<BF16>(y[j]), K - el(j));
    } else if constexpr (Q == Quant::MX) {
        // the 4 lanes of a block of 32 share an exponent; a block that holds a NaN or
        // an infinity has E8M0 255 and zero codes
        const bool fp4 = p.fp4_or_i8 != 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float m = amax8(y[j]);
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) bad |= (uint32_t)((__float_as_uint(y[j][i]) & 0x7F800000u) == 0x7F800000u);
            m = fmaxf(m, __shfl_xor(m, 1));
            m = fmaxf(m, __shfl_xor(m, 2));
            bad |= __shfl_xor(bad, 1);
            bad |= __shfl_xor(bad, 2);
            int e = 0;
            if (bad) {
                e = 255;
            } else if (m > 0.f) {
                e = (int)((__float_as_uint(m) >> 23) & 0xFFu) - (fp4 ? 2 : 8);
                e = e < 0 ? 0 : e;
            }
            if (el(j) >= K) continue;
            const int64_t at = row * K + el(j);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = e == 255 ? 0.f : ldexpf(y[j][i], 127 - e);
            if (fp4) {
                uint32_t q = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) q |= (e == 255 ? 0u : e2m1_of(y[j][i], v[i])) << (4 * i);
                *(uint32_t*)((char*)p.out + at / 2) = q;
            } else {
                *(uint2*)((char*)p.out + at) = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
            }
            if ((t & 3) == 0) ((uint8_t*)p.scale)[at / 32] = (uint8_t)e;
        }
    } else {
        const bool i8 = Q == Quant::TOKEN && p.fp4_or_i8 != 0;
        const float top = i8 ? 127.f : 448.f;
        float s = 1.f;
        if constexpr (Q == Quant::TOKEN) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) m = fmaxf(m, amax8(y[j]));
            m = row_reduce<TPR, true>(m, red[1]);
            s = scale_of(m, top);
            if (t == 0) ((float*)p.scale)[row] = s;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if constexpr (Q == Quant::BLOCK) {
                float m = amax8(y[j]);
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
                s = scale_of(m, top);
                if ((t & 15) == 0 && el(j) < K) ((float*)p.scale)[row * (K / 128) + el(j) / 128] = s;
            }
            const int n = K - el(j);
            if (n <= 0) continue;
            float v[8];
            divide8(y[j], s, top, v);
            uint2 q;
            if (i8) {
                q.x = int8_code(v[0]) | int8_code(v[1]) << 8 | int8_code(v[2]) << 16 | int8_code(v[3]) << 24;
                q.y = int8_code(v[4]) | int8_code(v[5]) << 8 | int8_code(v[6]) << 16 | int8_code(v[7]) << 24;
            } else {
                q = make_uint2(e4m3x4_below(v[0], v[1], v[2], v[3]), e4m3x4_below(v[4], v[5], v[6], v[7]));
            }
            uint8_t* o = (uint8_t*)p.out + row * K + el(j);
            if (VEC) {
                *(uint2*)o = q;
            } else if (n >= 8) {
                ((Any8*)o)->v = q;
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (i < n) o[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
            }
        }
    }
}

template <bool BF16, Quant Q, int TPR, int NV, bool VEC>
hipError_t go(const RowParams& p, hipStream_t st) {
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    hipLaunchKernelGGL((row_kernel<BF16, Q, TPR, NV, VEC>), dim3((unsigned)((p.rows + RPW - 1) / RPW)), dim3(TPR < 256 ? 256 : TPR), 0, st, p);
    return hipGetLastError();
}

// Threads of a row by its width.  One wave as long as its registers hold the row: no barrier
// for the sums (8191 rows, norm with a residual and scales of tokens, us: width 512 one wave
// 9.8, four 14.3; 1024 12.5, 19.1; 2048 21.6, 26.1), but SwiGLU, which has less to wait for and
// twice the input, from 1024 on four (2048, scales of blocks: 18.3, 16.3) unless it waits for a
// row's scale too (tokens: 17.5, 25.0).  Then four, eight or sixteen (4096: four
// 46.6, eight 54.8; 8192 four 85.7, eight 85.1, sixteen with a group each 1.5 times as long;
// 16384 four 178, eight 169, sixteen 171; SwiGLU 135, 138, 128).  Longer rows: sixteen with up to eight groups
// a thread, of which a row just above 16384 leaves most empty (residual, tokens: 512 of 65536 44, 5.3 TB/s;
// 2048 of 16384 43, 5.4; of 16512 62, 3.8).  Up to kFewRows rows the
// steps of a thread count, so it has as few groups as there is a variant for (norm with scales
// of blocks, on the card, 5 / 256 / 700 rows: 2048 one wave 5.1 / 6.0 / 6.4, four 3.2 / 3.7 /
// 4.4; 4096 four 4.1 / 4.6 / 6.3, eight 3.4 / 4.1 / 6.2; 8192 four 5.5 / 6.6 / 9.9, eight 4.2 /
// 5.4 / 9.4, sixteen 3.9 / 5.2 / 9.4).
constexpr int64_t kFewRows = 1024;
template <bool BF16, Quant Q>
hipError_t pick(const RowParams& p, bool vec, hipStream_t st) {
    const int K = p.width;
    if constexpr (Q == Quant::SAME16 || Q == Quant::TOKEN) {
        // (rows that start at any element: 8191 of 1999, 16-bit output, 24 us, of 2000 20; by
        // 2-byte loads that are consecutive over a wave 48)
        if (!vec) {
            if (K <= 2048) return go<BF16, Q, 64, 4, false>(p, st);
            if (K <= 8192) return go<BF16, Q, 512, 2, false>(p, st);
            return go<BF16, Q, 1024, 8, false>(p, st);
        }
    }
    const bool few = p.rows <= kFewRows;
    if (K <= 512) return go<BF16, Q, 64, 1, true>(p, st);
    if (K <= 1024 && !few) return go<BF16, Q, 64, 2, true>(p, st);
    if (K <= 2048) return (p.silu && Q != Quant::TOKEN) || few ? go<BF16, Q, 256, 1, true>(p, st) : go<BF16, Q, 64, 4, true>(p, st);
    if (K <= 4096) return few ? go<BF16, Q, 512, 1, true>(p, st) : go<BF16, Q, 256, 2, true>(p, st);
    if (K <= 8192) return go<BF16, Q, 512, 2, true>(p, st);
    if (K <= 16384) return go<BF16, Q, 1024, 2, true>(p, st);
    return go<BF16, Q, 1024, 8, true>(p, st);
}

}  // namespace

hipError_t row_launch(const RowArgs& a) {
    RowParams p{};
    p.x = a.x;
    p.res = a.res;
    p.w = a.w;
    p.sum = a.sum;
    p.out = a.out;
    p.scale = a.scale;
    p.rows = a.rows;
    p.x_stride = a.x_stride;
    p.res_stride = a.res_stride;
    p.sum_stride = a.sum_stride;
    p.width = a.width;
    p.eps = a.eps;
    p.w_offset = a.w_offset;
    p.silu = a.silu;
    p.w_f32 = a.w_f32;
    p.fp4_or_i8 = a.kind == RowOut::TOKEN_I8 || a.kind == RowOut::MX_F4;
    const bool vec = a.width % 8 == 0 && a.x_stride % 8 == 0 && (!a.res || a.res_stride % 8 == 0) && (!a.sum || a.sum_stride % 8 == 0);
    switch (a.kind) {
        case RowOut::SAME16: return a.bf16 ? pick<true, Quant::SAME16>(p, vec, a.stream) : pick<false, Quant::SAME16>(p, vec, a.stream);
        case RowOut::TOKEN_F8:
        case RowOut::TOKEN_I8: return a.bf16 ? pick<true, Quant::TOKEN>(p, vec, a.stream) : pick<false, Quant::TOKEN>(p, vec, a.stream);
        case RowOut::BLOCK_F8: return a.bf16 ? pick<true, Quant::BLOCK>(p, vec, a.stream) : pick<false, Quant::BLOCK>(p, vec, a.stream);
        default: return a.bf16 ? pick<true, Quant::MX>(p, vec, a.stream) : pick<false, Quant::MX>(p, vec, a.stream);
    }
}

}  // namespace hq
