// Routing to experts and the weighted sum of what they answer.
//
// hq_moe_route: per token, scores s_e = softmax_e(l) or 1 / (1 + e^-l_e), the
// values that rank the experts c_e = s_e + bias_e (without a bias the logits
// themselves, which order the experts alike), the best groups by the sum of their
// best members, the k best experts of those, and their weights.
//
// A choice is a whole number, and a rounding must not turn it: two experts whose fp32
// scores round to the same value still come in the order that the formula gives.  Doubles
// for every expert would do, and cost twice the instructions, which are what bounds the
// kernel (one wave per token, lane l holding the NE experts from NE l on).  So fp32
// values, whose errors have a bound, only rule out: a threshold is searched bit by bit on
// the scalar unit that k lanes' best values reach (the k best taken one after the other
// would be a reduction over the wave each); what lies below it by more than the bound is
// out, and the few others, little more than k, move to a lane each, get their value in
// 64 bits and are ranked by counting.  Groups whose order the bound leaves open are
// formed in 64 bits; a NaN, or more than 64 left, sends a token to a slow way.
#include "hq_device.hpp"
#include "hq_kv.h"
#include "hq_layer.h"
#include "layer_rows.hpp"

namespace hq {

namespace {

struct RouteParams {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t T, stride;
    int E, k, groups, top_groups, group_best;
    FastDiv per_group;  // experts of a group
    int in_lanes;       // lanes that hold a group, where it fills whole lanes, 1 2 4 8 or 16 of them (else 0)
    int dtype, sigmoid, renorm, wide;
    float scale;
};

constexpr double kLowest = -__builtin_huge_val();

// The value of lane `ctrl` says (DPP: no LDS), for reductions; every lane has a source.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)u) | ((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;  // (a mirror is a xor once its halves agree)

__device__ __forceinline__ double from_lane(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
// Over 16 lanes, and over the wave: within 16 lanes by DPP, the four rows' results by readlane.
__device__ __forceinline__ double row_sum(double v) {
    v += dpp<kXor1>(v);
    v += dpp<kXor2>(v);
    v += dpp<kMirror8>(v);
    return v + dpp<kMirror16>(v);
}
__device__ __forceinline__ double wave_sum(double v) {
    v = row_sum(v);
    return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<kXor1>(v));
    v = fmaxf(v, dpp<kXor2>(v));
    v = fmaxf(v, dpp<kMirror8>(v));
    v = fmaxf(v, dpp<kMirror16>(v));
    auto row = [&](int l) { return __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(v), l)); };
    return fmaxf(fmaxf(row(0), row(16)), fmaxf(row(32), row(48)));
}

// e^x for x <= 0 (NaN: NaN): x = n ln 2 + r, the Taylor series of e^r to r^12 (|r| <= 0.347:
// the rest is below 2^-52), scaled by 2^n; 20 instructions.
template <bool LOOP>
__device__ __forceinline__ double exp_neg(double x) {
    auto k = [](double v) {  // in a loop: the coefficients made anew, not kept in registers through it
        if constexpr (LOOP) asm volatile("" : "+s"(v));
        return v;
    };
    x = x < -1100.0 ? -1100.0 : x;
    const double n = rint(x * 1.4426950408889634);
    const double r = fma(-n, k(1.9082149292705877e-10), fma(-n, k(0.69314718036912382), x));  // ln 2 in two parts
    double p = k(1.0 / 479001600);
    p = fma(p, r, k(1.0 / 39916800));
    p = fma(p, r, k(1.0 / 3628800));
    p = fma(p, r, k(1.0 / 362880));
    p = fma(p, r, k(1.0 / 40320));
    p = fma(p, r, k(1.0 / 5040));
    p = fma(p, r, k(1.0 / 720));
    p = fma(p, r, k(1.0 / 120));
    p = fma(p, r, k(1.0 / 24));
    p = fma(p, r, k(1.0 / 6));
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}
// 1 / (1 + e^-x): from t = e^-|x| <= 1, so without overflow; 1 / (1 + t) by two steps of
// Newton's iteration.
template <bool LOOP>
__device__ __forceinline__ double sigmoid(double x) {
    const double t = exp_neg<LOOP>(-fabs(x)), d = 1.0 + t;
    double y = __builtin_amdgcn_rcp(d);
    y = fma(fma(-d, y, 1.0), y, y);
    y = fma(fma(-d, y, 1.0), y, y);
    return x < 0 ? t * y : y;
}

// 1 / x for normal x (v_rcp_f64 and two steps of Newton's iteration).
__device__ __forceinline__ double reciprocal(double x) {
    double y = __builtin_amdgcn_rcp(x);
    y = fma(fma(-x, y, 1.0), y, y);
    return fma(fma(-x, y, 1.0), y, y);
}

// NaN ranks with -inf.
__device__ __forceinline__ double rank_of(double x) { return x != x ? kLowest : x; }
// Unsigned integers in the order of the values (-0 as 0); every value's is above 0.
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
    return u ^ (uint64_t)((int64_t)u >> 63 | (int64_t)0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// What the ways to choose have in common: a token's logits, its scores in 64 bits.
struct Token {
    const RouteParams& p;
    int64_t t;
    float top;     // the largest logit (softmax)
    double inv;    // what scores are multiplied by: 1 / the sum over all experts, where it counts

    __device__ __forceinline__ float logit(int e) const {
        const int64_t at = t * p.stride + e;
        return p.dtype == HQ_DT_FP32   ? ((const float*)p.logits)[at]
               : p.dtype == HQ_DT_BF16 ? bits16_to_f32<true>(((const uint16_t*)p.logits)[at])
                                       : bits16_to_f32<false>(((const uint16_t*)p.logits)[at]);
    }
    template <bool LOOP = false>
    __device__ __forceinline__ double score(float x) const {  // not yet times inv
        if (p.sigmoid) return sigmoid<LOOP>((double)x);
        return top == -INFINITY && x == top ? 0.0 : exp_neg<LOOP>((double)x - (double)top);
    }
    // The weights of the chosen: lane `chosen` has score w (times inv) of expert e, rank r; the
    // token's lanes are a wave, or 16 (ROW).
    template <bool ROW = false>
    __device__ __forceinline__ void store(bool chosen, double w, int e, int r) const {
        w = chosen ? w : 0.0;
        if (p.renorm) {
            const double sum = ROW ? row_sum(w) : wave_sum(w);
            w = sum == 0 ? 0.0 : sum > 1e-290 ? w * reciprocal(sum) : w / sum;
        }
        if (chosen) {
            p.ids[t * p.k + r] = e;
            p.weights[t * p.k + r] = (float)(w * (double)p.scale);
        }
    }
};

// A token's few experts that are left, in their order, for a lane each; how many they are, and
// what the scores need.
struct Few {
    uint32_t expert[64];
    float logit[64], bias[64];
    int count;
    float top;
    double inv;
};

// What ranks expert e.
__device__ __forceinline__ double rank_value(const Token& tok, int e) {
    const float x = tok.logit(e);
    return rank_of(tok.p.bias ? tok.score<true>(x) * tok.inv + (double)tok.p.bias[e] : (double)x);
}

// Whether group lane / L stays, in 64 bits; L lanes to a group look at its members.
__device__ __forceinline__ bool group_stays(const Token& tok, int L) {
    const RouteParams& p = tok.p;
    const int lane = threadIdx.x & 63, S = (int)p.per_group.d, g = lane / L;
    double a = kLowest, b = kLowest;  // the two best, a >= b
    if (g < p.groups)
#pragma unroll 1
        for (int i = lane % L; i < S; i += L) {
            const int e = g * S + i;
            const double v = p.bias || p.group_best == 1 ? rank_value(tok, e) : rank_of(tok.score<true>(tok.logit(e)) * tok.inv);
            b = fmax(b, fmin(a, v));
            a = fmax(a, v);
        }
#pragma unroll 1
    for (int x = 1; x < L; x <<= 1) {
        const double a2 = __shfl_xor(a, x), b2 = __shfl_xor(b, x);
        b = fmax(fmin(a, a2), fmax(b, b2));
        a = fmax(a, a2);
    }
    const double value = p.group_best == 2 ? rank_of(a + b) : a;
    int better = 0;  // fewer than top_groups are better than one that stays (of equals the lower is)
#pragma unroll 1
    for (int o = 0; o < p.groups; ++o) {
        const double v = from_lane(value, o * L);
        better += v > value || (v == value && o < g) ? 1 : 0;
    }
    return better < p.top_groups && g < p.groups;
}
__device__ __forceinline__ int lanes_of_group(int groups) {
    int L = 64;
    while (L > 1 && L * groups > 64) L >>= 1;
    return L;
}

// The slow way: everything in 64 bits, formed anew wherever it is looked at; the k best one
// after the other.
__device__ __forceinline__ void route_slowly(const Token& tok) {
    const RouteParams& p = tok.p;
    const int lane = threadIdx.x & 63, L = lanes_of_group(p.groups);
    const uint64_t stay = p.groups > 1 ? __ballot(group_stays(tok, L)) : ~0ull;
    uint64_t taken = 0;  // bit i: expert 64 i + lane
    int my_id = 0;
#pragma unroll 1
    for (int r = 0; r < p.k; ++r) {
        double best = kLowest;
        int at = 1 << 20;
#pragma unroll 1
        for (int i = 0, e = lane; e < p.E; ++i, e += 64) {
            if (((taken >> i) & 1) || (p.groups > 1 && !((stay >> (p.per_group.div(e) * L)) & 1))) continue;
            const double v = rank_value(tok, e);
            if (v > best || at == 1 << 20) {
                best = v;
                at = e;
            }
        }
        // the largest, the lowest expert of equals (one is always left: k is at most the
        // experts of the groups that stay)
#pragma unroll 1
        for (int x = 32; x > 0; x >>= 1) {
            const double v = __shfl_xor(best, x);
            const int o = __shfl_xor(at, x);
            const bool is = (o < 1 << 20) && (at == 1 << 20 || v > best || (v == best && o < at));
            best = is ? v : best;
            at = is ? o : at;
        }
        if (at % 64 == lane) taken |= 1ull << (at / 64);
        if (lane == r) my_id = at;
    }
    tok.store(lane < p.k, lane < p.k ? tok.score<true>(tok.logit(my_id)) * tok.inv : 0.0, my_id, lane);
}

// The quick way as far as the few that are left; their number, or 0 where it cannot tell.
template <int NE>
__device__ __forceinline__ int rule_out(const RouteParams& p, Token& tok, float* members, Few& few) {
    const int lane = threadIdx.x & 63, E = p.E, e0 = lane * NE;
    const int64_t t = tok.t;

    float l[NE], bias[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        l[i] = -INFINITY;
        bias[i] = 0.f;
    }
    if (NE % 4 == 0 && p.wide && e0 < E) {  // fp32 rows of whole 16 bytes
#pragma unroll
        for (int i = 0; i < NE / 4; ++i) {
            if (e0 + 4 * i >= E) break;
            const v4f v = *(const v4f*)((const float*)p.logits + t * p.stride + e0 + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) l[(4 * i + j) % NE] = v[j];
            if (p.bias) {
                const v4f b = *(const v4f*)(p.bias + e0 + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) bias[(4 * i + j) % NE] = b[j];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (e0 + i < E) {
                l[i] = tok.logit(e0 + i);
                if (p.bias) bias[i] = p.bias[e0 + i];
            }
    }
    // a NaN among the logits, seen in their sum (so are infinities of both signs: a token that
    // has them goes the slow way)
    float all = l[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) all += l[i];
    const uint64_t odd = __ballot(all != all);
    // Scores.  Softmax in 64 bits, where the sum over all experts counts (where the weights are
    // renormalised and nothing else asks, it cancels).  Sigmoid: e^-|l| and 1 / (1 + e^-|l|)
    // from the hardware's exp2 and reciprocal (each off by one unit of fp32, the argument
    // by 2^-24 of itself, which t = e^-|l| makes less than 2^-24 again): within 2^-21.
    const bool pairs = p.groups > 1 && p.group_best == 2, scored = p.bias || pairs;
    float c[NE];  // ranking values
    if (!p.sigmoid) {
        float top = l[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) top = fmaxf(top, l[i]);
        tok.top = wave_max(top);
        if (scored || !p.renorm) {
            double s[NE], sum = 0;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                s[i] = tok.score(l[i]);
                sum += e0 + i < E ? s[i] : 0.0;
            }
            sum = wave_sum(sum);
            tok.inv = sum == 0 ? 0.0 : 1.0 / sum;  // (every logit -inf: weights 0)
#pragma unroll
            for (int i = 0; i < NE; ++i) c[i] = (float)(s[i] * tok.inv);
        }
        if (odd) {  // a NaN is in every weight
            bool nan = false;
#pragma unroll
            for (int i = 0; i < NE; ++i) nan = nan || l[i] != l[i];
            if (__ballot(nan)) tok.inv = __builtin_nan("");
        }
    } else if (scored) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float x = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(l[i])), y = __builtin_amdgcn_rcpf(1.0f + x);
            c[i] = l[i] < 0 ? x * y : y;
        }
    }
    // How far c may be off: scores by 2^-20, the sum with a bias by 2^-24 of itself.
    auto off = [&](float v) { return p.bias ? 0x1p-19f + 0x1p-22f * fabsf(v) : 0.f; };
    uint32_t key[NE];  // in the order of the ranking, 0 for what cannot be taken
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        if (p.bias) c[i] += bias[i];
        else if (!pairs) c[i] = l[i];
        key[i] = ordered(p.bias ? c[i] : l[i]);
    }
    if (E < 64 * NE) {
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = e0 + i < E ? key[i] : 0;
    }
    if (p.bias) {
        all = c[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) all += c[i];
        if (__ballot(all != all)) return 0;
    } else if (odd) {
        return 0;
    }

    if (p.groups > 1) {
        // the value of a group: the sum of its best one or two; L lanes to a group
        const int S = (int)p.per_group.d;
        int L = p.in_lanes;
        float a = -INFINITY, b = -INFINITY;  // the two best, a >= b
        auto take = [&](float v) {
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
        };
        if (L) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (e0 + i < E) take(c[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (e0 + i < E) members[e0 + i] = c[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            L = lanes_of_group(p.groups);
            const int g = lane / L;
            if (g < p.groups)
                for (int i = lane % L; i < S; i += L) take(members[g * S + i]);
        }
        auto join = [&](float a2, float b2) {
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
        };
        if (L > 1) join(dpp<kXor1>(a), dpp<kXor1>(b));
        if (L > 2) join(dpp<kXor2>(a), dpp<kXor2>(b));
        if (L > 4) join(dpp<kMirror8>(a), dpp<kMirror8>(b));
        if (L > 8) join(dpp<kMirror16>(a), dpp<kMirror16>(b));
        for (int x = 16; x < L; x <<= 1) join(__shfl_xor(a, x), __shfl_xor(b, x));
        // A group stays where fewer than top_groups are better (of equals the lower is).  Values
        // with errors: where it is sure whether so many are.  (The sum of two: both errors, and
        // 2^-24 of the sum.)
        const float value = pairs ? a + b : a;
        const float err = scored ? 0x1p-17f + 0x1p-20f * (fabsf(a) + (pairs ? fabsf(b) : 0.f)) : 0.f;
        const float low = value - err, high = value + err;
        const int g = lane / L, x = lane % L;
        int sure = 0, maybe = 0;
        const uint64_t mask = L == 64 ? ~0ull : (1ull << L) - 1;
        for (int o = 0; o < p.groups; o += L) {  // lane x of each group looks at group o + x
            const int other = o + x;
            const float low_o = __shfl(low, other * L), high_o = __shfl(high, other * L);
            const bool is = other < p.groups && other != g;
            const bool s = is && (low_o > high || (!scored && low_o == high && other < g));
            const bool m = scored ? is && high_o >= low : s;
            sure += __popcll(__ballot(s) >> (lane - x) & mask);
            maybe += __popcll(__ballot(m) >> (lane - x) & mask);
        }
        bool stays = maybe < p.top_groups && g < p.groups;
        const bool open = g < p.groups && ((!stays && sure < p.top_groups) || (scored && !(err < INFINITY)));
        if (__ballot(open)) stays = group_stays(tok, L);
        if (p.in_lanes) {
#pragma unroll
            for (int i = 0; i < NE; ++i) key[i] = stays ? key[i] : 0;
        } else {
            const uint64_t stay = __ballot(stays);
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (e0 + i < E && !((stay >> (p.per_group.div(e0 + i) * L)) & 1)) key[i] = 0;
        }
    }

    // a threshold that at least k lanes' best keys reach, and few more (fewer than k lanes: 0)
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) best = max(best, key[i]);
    uint32_t bar = 0;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
        const int n = __popcll(__ballot(best >= (bar | bit)));
        if (n >= p.k) {
            bar |= bit;
            if (n <= p.k + 2) break;
        }
    }
    // The k-th best value is at least the threshold less an error, so what comes out two errors
    // below is not among them.  (bar can be 0, or a NaN's key: then everything is above.)
    if (p.bias) {
        const float v = value_of(bar), w = v - 2 * off(v);
        bar = w == w ? ordered(w) : 0;
    }
    bar = max(bar, 1u);
    int before = 0, total = 0;  // picked experts of the lanes before, of all
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const uint64_t m = __ballot(key[i] >= bar);
        before = __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, before));
        total += __popcll(m);
    }
    if (total > 64) return 0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (key[i] >= bar) {
            few.expert[before] = (uint32_t)(e0 + i);
            few.logit[before] = l[i];
            if (p.bias) few.bias[before] = bias[i];
            ++before;
        }
    return total;
}

// ... and their order: the value of each in 64 bits, its rank by counting the larger ones; of
// equal upper halves the lower count too.  Lane by lane of the wave, `total` of them, ...
__device__ __forceinline__ void rank_few(const Token& tok, const Few& few, int total) {
    const RouteParams& p = tok.p;
    const int lane = threadIdx.x & 63;
    const float x = few.logit[lane];
    const double s = tok.score(x) * tok.inv;
    const uint64_t full = p.bias ? ordered(s + (double)few.bias[lane]) : (uint64_t)ordered(x) << 32;
    const uint32_t k = lane < total ? (uint32_t)(full >> 32) : 0;  // (0: below every value's)
    int rank = 0;
    uint64_t equal = 0;  // lanes that have another's upper half
    for (int j = 0; j < total; ++j) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)k, j);
        rank += o > k ? 1 : 0;
        equal |= __ballot(o == k) & ~(1ull << j);
    }
    if (equal) {
        rank = 0;
        for (int j = 0; j < total; ++j) {
            const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(full >> 32), j) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)full, j);
            rank += o > full || (o == full && j < lane) ? 1 : 0;
        }
    }
    tok.store(lane < total && rank < p.k, s, (int)few.expert[lane], rank);
}
// ... or, where a token has up to 16, four tokens in one wave, 16 lanes each: the others of a row
// come by its rotation.
template <int N>
__device__ __forceinline__ void compare(uint64_t full, bool whole, int lane, int& rank, bool& equal) {
    const uint32_t hi = (uint32_t)(full >> 32), lo = (uint32_t)full, o_hi = dpp<0x120 + N>(hi);  // row_ror:N
    if (whole) {
        const uint64_t o = (uint64_t)o_hi << 32 | dpp<0x120 + N>(lo);
        rank += o > full || (o == full && ((lane - N) & 15) < (lane & 15)) ? 1 : 0;
    } else {
        rank += o_hi > hi ? 1 : 0;
        equal = equal || o_hi == hi;
    }
    if constexpr (N < 15) compare<N + 1>(full, whole, lane, rank, equal);
}
__device__ __forceinline__ void rank_rows(const RouteParams& p, int64_t first, const Few (&few)[4]) {
    const int lane = threadIdx.x & 63, w = lane >> 4, i = lane & 15;
    const Few& f = few[w];
    const int total = f.count;
    const Token tok{p, first + w, f.top, f.inv};
    const float x = f.logit[i];
    const double s = tok.score(x) * tok.inv;
    uint64_t full = p.bias ? ordered(s + (double)f.bias[i]) : (uint64_t)ordered(x) << 32;
    full = i < total ? full : (uint64_t)i;  // (below every value's, and different)
    int rank = 0;
    bool equal = false;
    compare<1>(full, false, lane, rank, equal);
    if (__ballot(equal && i < total)) {
        rank = 0;
        compare<1>(full, true, lane, rank, equal);
    }
    tok.store<true>(i < total && rank < p.k, s, (int)f.expert[i], rank);
}

// A wave to a token as far as the few; then one wave for the four tokens of a workgroup (which
// one goes round, so that no SIMD has them all): ranking and weights in 64 bits are a third of
// the instructions, and a token's few fill a quarter of a wave.  16384 tokens, 256 experts in
// 8 groups, biased sigmoid scores: 13.7 us, each wave to the end for its own token 16.4; what
// is left is the vector instructions' issue (some 340 a token, 9 us) and the launch.
template <int NE>
__global__ __launch_bounds__(256) void route_kernel(RouteParams p) {
    extern __shared__ float members[];  // [4 waves][E], for groups that do not fill whole lanes
    __shared__ Few few[4];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Token tok{p, (int64_t)blockIdx.x * 4 + wave, 0.f, 1.0};
    int total = 0;
    if (tok.t < p.T) {
        total = rule_out<NE>(p, tok, members + (int64_t)wave * p.E, few[wave]);
        if (total == 0) {
            route_slowly(tok);
        } else if (total > 16) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            rank_few(tok, few[wave], total);
            total = 0;
        }
    }
    if ((threadIdx.x & 63) == 0) {
        few[wave].count = total;
        few[wave].top = tok.top;
        few[wave].inv = tok.inv;
    }
    __syncthreads();
    if (wave == (int)(blockIdx.x & 3)) rank_rows(p, (int64_t)blockIdx.x * 4, few);
}

template <int NE>
hipError_t go(RouteParams p, hipStream_t st) {
    const int S = p.E / p.groups, lanes = S / NE;
    p.in_lanes = S % NE == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    const size_t lds = p.groups > 1 && !p.in_lanes ? (size_t)p.E * 4 * sizeof(float) : 0;
    // Above 64 KB in all (some 3900 experts and up, in groups that fill no whole lanes) LDS is asked for, at
    // each call: it is granted for a kernel on one device, the current one.
    if (lds + 4 * sizeof(Few) > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)route_kernel<NE>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((route_kernel<NE>), dim3((unsigned)((p.T + 3) / 4)), dim3(256), lds, st, p);
    return hipGetLastError();
}

// ---- the weighted sum ----

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// place[p] = the row that holds pair p (rows sorted by expert).
__global__ __launch_bounds__(256) void place_kernel(const int32_t* __restrict__ sorted, int64_t P, int32_t* __restrict__ place) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= P) return;
    const int32_t p = sorted[i];
    if (p >= 0 && p < P) place[p] = (int32_t)i;
}

// Up to so many pairs, each token's workgroup looks through `sorted` for its rows itself: a
// launch less (8 experts, 7168 columns, 5 tokens: 4.9 us, with a launch for the places
// 7.9; 100 tokens: 6.7, 7.9).
constexpr int kCombineFew = 1024;

struct CombineParams {
    const uint16_t *y, *add;
    const float* weights;
    const int32_t *sorted, *place;  // place NULL: of few pairs
    uint16_t* out;
    int64_t N, P;
    int k;
};

// out[t] = rnd16(add[t] + sum_j w[t][j] y[row(t, j)]), j in order, fp32.  Bound by HBM, so
// what matters is how many loads are on their way: a workgroup takes a token, its lanes
// look up the token's rows side by side, and a thread then has the loads of eight rows
// under way at a time, 8 columns each (of which `cols` are the row's).  A row of weight 0 is
// not read.  4095 tokens of 8 rows, us: 7168 columns 99 (5.9 TB/s; where each call has new rows 114,
// 5.2), 7169 120, 1776 26.7, 1777 34.2 (by single columns 45.4).
template <bool BF16, bool VEC, bool NT, int R>
__device__ __forceinline__ void add_rows(const CombineParams& p, uint64_t& left, int64_t row, float w, int64_t n, int cols, float (&acc)[8]) {
    v4u v[R];
    float wj[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {  // the next R rows that count
        const int j = __builtin_ctzll(left);
        left &= left - 1;
        const int64_t at = (int64_t)__builtin_amdgcn_readlane((int)row, j);
        wj[r] = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(w), j));
        v[r] = load8<VEC, NT>(p.y + at * p.N + n, cols);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float y[8];
        unpack8<BF16>(v[r], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += wj[r] * y[i];
    }
}

template <bool BF16, bool VEC, bool NT>
__global__ __launch_bounds__(512) void combine_kernel(CombineParams p) {
    constexpr int C = 8;
    __shared__ int row_of[kCombineFew];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63;
    if (p.sorted && !p.place) {  // (then k is at most kCombineFew)
        for (int j = threadIdx.x; j < p.k; j += blockDim.x) row_of[j] = -1;
        __syncthreads();
        for (int i = threadIdx.x; i < p.P; i += blockDim.x) {
            const int64_t j = p.sorted[i] - t * p.k;
            if (j >= 0 && j < p.k) row_of[j] = i;
        }
        __syncthreads();
    }
    // the token's first 64 pairs: lane j's row (each wave for itself)
    float w0 = 0.f;
    int64_t row0 = 0;
    auto look = [&](int j0, float& w, int64_t& row) -> uint64_t {
        const int j = j0 + lane;
        bool have = j < p.k;
        const int64_t pair = t * p.k + (have ? j : 0);
        w = have ? p.weights[pair] : 0.f;
        row = pair;
        have = have && w != 0.f;
        if (p.sorted && !p.place) {
            row = have ? row_of[j] : -1;
            have = row >= 0;
        } else if (p.sorted) {
            // a pair that no row names has whatever the workspace held: it counts only if
            // its row names it
            row = p.place[pair];
            const bool in = row >= 0 && row < p.P;
            have = have && in && p.sorted[in ? row : 0] == (int32_t)pair;
        }
        return __ballot(have);
    };
    const uint64_t have0 = look(0, w0, row0);
    for (int64_t n0 = (int64_t)blockIdx.y * blockDim.x; n0 * C < p.N; n0 += (int64_t)gridDim.y * blockDim.x) {
        const int64_t n = (n0 + threadIdx.x) * C;
        const bool live = n < p.N;
        const int64_t nl = live ? n : 0;  // (past the row: its start, not stored)
        const int cols = VEC ? 8 : (int)min(p.N - nl, (int64_t)8);
        float a[8], acc[8] = {};
        unpack8<BF16>(p.add ? load8<VEC>(p.add + t * p.N + nl, cols) : v4u{0, 0, 0, 0}, a);
        for (int j0 = 0; j0 < p.k; j0 += 64) {
            float w = w0;
            int64_t row = row0;
            uint64_t left = j0 ? look(j0, w, row) : have0;
            while (__popcll(left) >= 8) add_rows<BF16, VEC, NT, 8>(p, left, row, w, nl, cols, acc);
            if (__popcll(left) >= 4) add_rows<BF16, VEC, NT, 4>(p, left, row, w, nl, cols, acc);
            if (__popcll(left) >= 2) add_rows<BF16, VEC, NT, 2>(p, left, row, w, nl, cols, acc);
            if (left) add_rows<BF16, VEC, NT, 1>(p, left, row, w, nl, cols, acc);
        }
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += a[i];
        store8<VEC>(p.out + t * p.N + n, pack8<BF16>(acc), cols);
    }
}

// (rows of 4-byte scales: 32760 of 14 words 4.8 us, of 57 6.2, 800 of 56 4.8: the launch)
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
    p.per_group = FastDiv::of((uint32_t)(a.experts / a.groups));
    p.wide = a.dtype == HQ_DT_FP32 && a.stride % 4 == 0 && a.experts % 4 == 0;
    p.dtype = a.dtype;
    p.sigmoid = a.sigmoid;
    p.renorm = a.renorm;
    p.scale = a.scale;
    // As many experts a lane as there are lanes' worth.  16384 tokens, biased sigmoid, us: 1024 experts 20, 1025 294,
    // 2048 209, 4096 201: 64 a lane take 256 registers, so one wave a SIMD (and 1025 no wide loads).
    if (a.experts <= 64) return go<1>(p, a.stream);
    if (a.experts <= 128) return go<2>(p, a.stream);
    if (a.experts <= 256) return go<4>(p, a.stream);
    if (a.experts <= 512) return go<8>(p, a.stream);
    if (a.experts <= 1024) return go<16>(p, a.stream);
    return go<64>(p, a.stream);
}

hipError_t combine_launch(const CombineArgs& a) {
    const int64_t P = a.T * a.top_k;
    const bool few = P <= kCombineFew;
    if (a.sorted && !few) {
        hipLaunchKernelGGL(place_kernel, dim3((unsigned)((P + 255) / 256)), dim3(256), 0, a.stream, a.sorted, P, a.place);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    CombineParams p{(const uint16_t*)a.y, (const uint16_t*)a.add, a.weights, a.sorted, few ? nullptr : a.place, (uint16_t*)a.out, a.N, P, a.top_k};
    const bool vec = a.N % 8 == 0;
    // a workgroup for a token, of as many threads as share its columns evenly; for few
    // tokens, which do not fill the chip, one for each 128 threads' columns (7168 columns, 5
    // tokens: 3.2 us, one workgroup each 4.6; 60: 3.7, 4.9)
    // (workgroups times threads stay below 2^32)
    const int64_t units = ceil_div(a.N, 8), turns = ceil_div(units, a.T < 1 << 23 ? 512 : 256);
    const int threads = a.T < 64 ? 128 : (int)ceil_div(ceil_div(units, turns), 64) * 64;
    const dim3 grid((unsigned)a.T, (unsigned)(a.T < 64 ? ceil_div(units, threads) : 1)), block(threads);
    // Rows that the 256 MB behind the L2s cannot hold go past them (y of 470 MB: 99 us, loaded
    // as others are 122; of 115 MB, just written: 29, 26)
    const bool nt = P * a.N * 2 > (int64_t)256 << 20;
    auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, a.stream, p); };
    if (a.bf16 && vec) launch(nt ? combine_kernel<true, true, true> : combine_kernel<true, true, false>);
    else if (a.bf16) launch(nt ? combine_kernel<true, false, true> : combine_kernel<true, false, false>);
    else if (vec) launch(nt ? combine_kernel<false, true, true> : combine_kernel<false, true, false>);
    else launch(nt ? combine_kernel<false, false, true> : combine_kernel<false, false, false>);
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
