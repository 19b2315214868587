// Routing to experts and the weighted sum of what they answer.
//
// hq_moe_route: per token, scores s_e = softmax_e(l) or 1 / (1 + e^-l_e), the
// values that rank the experts c_e = s_e + bias_e (without a bias the logits
// themselves, which order the experts alike), the best groups by the sum of their
// best members, the k best experts of those, and their weights.
//
// One wave per token, expert e = 64 i + lane of the wave.  Ranking values are
// doubles: two experts whose fp32 scores round to the same value still come in
// the order that the formula gives (a choice is a whole number, and a rounding
// must not turn it).  v_max_f64 runs at the rate of v_max_f32 here.
#include "hq_device.hpp"
#include "hq_layer.h"

namespace hq {

namespace {

struct RouteParams {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t T, stride;
    int E, k, groups, top_groups, group_best;
    int dtype, sigmoid, renorm;
    float scale;
};

constexpr double kLowest = -__builtin_huge_val();

__device__ __forceinline__ double shfl_xor_d(double v, int m) { return __shfl_xor(v, m); }

// The order-preserving key of x as an unsigned: NaN is the lowest, -0 equals 0.
// (Infinities keep their places: a bias of -inf ranks behind every number.)
__device__ __forceinline__ double rank_of(double x) { return x != x ? kLowest : x; }

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v = fmax(v, shfl_xor_d(v, m));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += shfl_xor_d(v, m);
    return v;
}

template <int NE>
__global__ __launch_bounds__(256) void route_kernel(RouteParams p) {
    extern __shared__ double members[];  // [4 waves][E], with groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= p.T) return;  // whole waves; no barrier below
    const int E = p.E;

    float l[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 64 * i + lane;
        l[i] = -INFINITY;
        if (e < E) {
            const int64_t at = t * p.stride + e;
            l[i] = p.dtype == HQ_DT_FP32   ? ((const float*)p.logits)[at]
                   : p.dtype == HQ_DT_BF16 ? bits16_to_f32<true>(((const uint16_t*)p.logits)[at])
                                           : bits16_to_f32<false>(((const uint16_t*)p.logits)[at]);
        }
    }
    // scores: sigmoid from e^-|l| <= 1; softmax less the largest logit
    double s[NE];
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const double x = l[i], e = exp(-fabs(x));
            s[i] = (x >= 0 ? 1.0 : e) / (1.0 + e);
        }
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) m = fmaxf(m, l[i]);
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
        double sum = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = m == -INFINITY && l[i] == m ? 0.0 : exp((double)l[i] - (double)m);
            sum += s[i];
        }
        sum = wave_sum(sum);
        const double inv = sum == 0 ? 0.0 : 1.0 / sum;  // (every logit -inf: weights 0)
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] *= inv;
    }
    double c[NE];
    uint64_t open = 0;  // bit i: expert 64 i + lane may still be taken
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 64 * i + lane;
        c[i] = p.bias ? s[i] + (double)(e < E ? p.bias[e] : 0.f) : (double)l[i];
        c[i] = rank_of(c[i]);
        if (e < E) open |= 1ull << i;
    }

    if (p.groups > 1) {
        // the value of a group: the sum of its best one or two ranking values (scores,
        // where there is no bias).  64 / L groups at a time, L lanes to a group.
        const int S = E / p.groups;
        double* mine = members + (int64_t)wave * E;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (64 * i + lane < E) mine[64 * i + lane] = p.bias ? c[i] : rank_of(s[i]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        int L = 64;
        while (L > 1 && L * p.groups > 64) L >>= 1;
        const int g = lane / L;
        double a = kLowest, b = kLowest;  // the two best, a >= b
        if (g < p.groups)
            for (int i = lane % L; i < S; i += L) {
                const double v = mine[g * S + i];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
        for (int x = 1; x < L; x <<= 1) {
            const double a2 = shfl_xor_d(a, x), b2 = shfl_xor_d(b, x);
            b = fmax(fmin(a, a2), fmax(b, b2));
            a = fmax(a, a2);
        }
        const double value = p.group_best == 2 ? rank_of(a + b) : a;
        // groups that stay: fewer than top_groups are better (the lower of equals is)
        int better = 0;
        for (int o = 0; o < p.groups; ++o) {
            const double v = __shfl(value, o * L);
            better += v > value || (v == value && o < g) ? 1 : 0;
        }
        const uint64_t stay = __ballot(better < p.top_groups && g < p.groups);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = 64 * i + lane;
            if (e < E && !((stay >> (e / S * L)) & 1)) open &= ~(1ull << i);
        }
    }

    // the k best: of the lanes' best values the largest, the lowest expert of equals
    int32_t* ids = p.ids + t * p.k;
    int my_id = 0;
    double my_s = 0, total = 0;
    for (int r = 0; r < p.k; ++r) {
        double best = kLowest;
        int at = 1 << 20;  // the lane's lowest open expert with that value
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const bool is = ((open >> i) & 1) && (c[i] > best || at == 1 << 20);
            best = is ? c[i] : best;
            at = is ? 64 * i + lane : at;
        }
        const double top = wave_max(best);
        int win = best == top ? at : 1 << 20;
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) win = min(win, __shfl_xor(win, x));
        // (an open expert is always left: k is at most the experts of the groups that stay)
        double score = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (i == win / 64) score = s[i];
        score = __shfl(score, win & 63);
        if ((win & 63) == lane) open &= ~(1ull << (win >> 6));
        total += score;
        if (lane == r) {
            my_id = win;
            my_s = score;
        }
    }
    if (lane < p.k) {
        double w = my_s;
        if (p.renorm) w = total == 0 ? 0.0 : w / total;
        ids[lane] = my_id;
        p.weights[t * p.k + lane] = (float)(w * (double)p.scale);
    }
}

template <int NE>
hipError_t go(const RouteParams& p, hipStream_t st) {
    const size_t lds = p.groups > 1 ? (size_t)p.E * 4 * sizeof(double) : 0;
    static const hipError_t attr = hipFuncSetAttribute((const void*)route_kernel<NE>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                                       64 * NE * 4 * (int)sizeof(double));
    if (attr != hipSuccess) return attr;
    hipLaunchKernelGGL((route_kernel<NE>), dim3((unsigned)((p.T + 3) / 4)), dim3(256), lds, st, p);
    return hipGetLastError();
}

// ---- the weighted sum ----

// place[p] = the row that holds pair p (rows sorted by expert).
__global__ __launch_bounds__(256) void place_kernel(const int32_t* __restrict__ sorted, int64_t P, int32_t* __restrict__ place) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= P) return;
    const int32_t p = sorted[i];
    if (p >= 0 && p < P) place[p] = (int32_t)i;
}

struct CombineParams {
    const uint16_t *y, *add;
    const float* weights;
    const int32_t *sorted, *place;
    uint16_t* out;
    int64_t N, P;
    int k;
};

// out[t] = rnd16(add[t] + sum_j w[t][j] y[row(t, j)]), j in order, fp32.  Bound by HBM:
// a thread sums 8 columns (VEC: 16-byte loads) over the token's rows.  A row of
// weight 0 is not read.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(CombineParams p) {
    const int64_t t = blockIdx.x;
    const int64_t n = ((int64_t)blockIdx.y * 256 + threadIdx.x) * (VEC ? 8 : 1);
    constexpr int C = VEC ? 8 : 1;
    float acc[C] = {};
    if (n >= p.N) return;
    for (int j = 0; j < p.k; ++j) {
        const int64_t pair = t * p.k + j;
        const float w = p.weights[pair];
        int64_t row = pair;
        bool have = w != 0.f;
        if (p.sorted) {
            // a pair that no row names has whatever the workspace held: it counts only if
            // its row names it
            row = p.place[pair];
            have = have && row >= 0 && row < p.P && p.sorted[row] == (int32_t)pair;
        }
        if (!have) continue;
        if constexpr (VEC) {
            const v4u v = ld16(p.y + row * p.N + n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = v[i];
                acc[2 * i] += w * bits16_to_f32<BF16>((uint16_t)u);
                acc[2 * i + 1] += w * bits16_to_f32<BF16>((uint16_t)(u >> 16));
            }
        } else {
            acc[0] += w * bits16_to_f32<BF16>(p.y[row * p.N + n]);
        }
    }
    if constexpr (VEC) {
        v4u o = p.add ? ld16(p.add + t * p.N + n) : v4u{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = o[i];
            const float a = acc[2 * i] + bits16_to_f32<BF16>((uint16_t)u), b = acc[2 * i + 1] + bits16_to_f32<BF16>((uint16_t)(u >> 16));
            o[i] = (uint32_t)f32_to_16<BF16>(a) | ((uint32_t)f32_to_16<BF16>(b) << 16);
        }
        *(v4u*)(p.out + t * p.N + n) = o;
    } else {
        p.out[t * p.N + n] = f32_to_16<BF16>(acc[0] + (p.add ? bits16_to_f32<BF16>(p.add[t * p.N + n]) : 0.f));
    }
}

__global__ __launch_bounds__(256) void gather_words_kernel(const uint32_t* __restrict__ A, const int* __restrict__ sorted, int64_t P, int top_k,
                                                           int64_t words, uint32_t* __restrict__ out) {
    const int64_t total = P * words;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / words, u = i - r * words;
        const int64_t pair = sorted[r] < 0 ? 0 : sorted[r] < P ? sorted[r] : P - 1;  // never outside A
        out[i] = A[pair / top_k * words + u];
    }
}

}  // namespace

hipError_t route_launch(const RouteArgs& a) {
    RouteParams p{};
    p.logits = a.logits;
    p.bias = a.bias;
    p.ids = a.ids;
    p.weights = a.weights;
    p.T = a.T;
    p.stride = a.stride;
    p.E = a.experts;
    p.k = a.top_k;
    p.groups = a.groups;
    p.top_groups = a.top_groups;
    p.group_best = a.group_best;
    p.dtype = a.dtype;
    p.sigmoid = a.sigmoid;
    p.renorm = a.renorm;
    p.scale = a.scale;
    if (a.experts <= 64) return go<1>(p, a.stream);
    if (a.experts <= 128) return go<2>(p, a.stream);
    if (a.experts <= 256) return go<4>(p, a.stream);
    if (a.experts <= 512) return go<8>(p, a.stream);
    if (a.experts <= 1024) return go<16>(p, a.stream);
    return go<64>(p, a.stream);
}

hipError_t combine_launch(const CombineArgs& a) {
    const int64_t P = a.T * a.top_k;
    if (a.sorted) {
        hipLaunchKernelGGL(place_kernel, dim3((unsigned)((P + 255) / 256)), dim3(256), 0, a.stream, a.sorted, P, a.place);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    CombineParams p{(const uint16_t*)a.y, (const uint16_t*)a.add, a.weights, a.sorted, a.place, (uint16_t*)a.out, a.N, P, a.top_k};
    const bool vec = a.N % 8 == 0;
    const dim3 grid((unsigned)a.T, (unsigned)((a.N + (vec ? 2047 : 255)) / (vec ? 2048 : 256)));
    if (vec && a.bf16) hipLaunchKernelGGL((combine_kernel<true, true>), grid, dim3(256), 0, a.stream, p);
    else if (vec) hipLaunchKernelGGL((combine_kernel<false, true>), grid, dim3(256), 0, a.stream, p);
    else if (a.bf16) hipLaunchKernelGGL((combine_kernel<true, false>), grid, dim3(256), 0, a.stream, p);
    else hipLaunchKernelGGL((combine_kernel<false, false>), grid, dim3(256), 0, a.stream, p);
    return hipGetLastError();
}

hipError_t gather_words_launch(const void* A, const int* sorted, int64_t P, int top_k, int64_t words, void* out, hipStream_t st) {
    int64_t blocks = (P * words + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    if (blocks < 1) return hipSuccess;
    hipLaunchKernelGGL(gather_words_kernel, dim3((unsigned)blocks), dim3(256), 0, st, (const uint32_t*)A, sorted, P, top_k, words, (uint32_t*)out);
    return hipGetLastError();
}

}  // namespace hq
