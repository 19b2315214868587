// Attention over a paged key/value cache behind a shared prefix.
//
// For a query row x (one token, one query head) and the keys j it sees,
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = log2(e) c(scale x.k_j).
// A part of the keys gives (m, l = sum p, O = sum p v), and parts are joined by
// M = max m, sum 2^(m - M) O / sum 2^(m - M) l, so the keys may be cut anywhere:
// between the prefix, which all rows of a key head read together as one tall
// matrix product, and each request's own keys, and again along a long axis
// where there are too few rows to fill the card.
//
// One workgroup takes a tile of rows and a part of the keys.  Rows of a key head
// are its tokens times the query heads that share it, so decoding batches still
// fill matrix tiles.  Per tile of keys: S^T = K Q^T with the queries along the
// columns, so a lane holds many keys of one query and the row statistics need
// one exchange between the two half-waves; P^T then is the right operand of
// O^T += V^T P^T as it lies in the registers, with V^T read by transposing LDS
// loads in the key order that S^T left.
#include "hq_device.hpp"
#include "hq_internal.h"
#include "hq_kv.h"

namespace hq {

namespace {

typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;
typedef __attribute__((address_space(3))) v2i* lds_v2i;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) v4f lds_v4f;

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 32;                       // query rows of a wave's matrix tile
constexpr int kFewTiles = 2;                    // tiles of kCols rows up to which a request counts as few rows
constexpr int kRowsWide = kWaves * kCols;       // rows of a workgroup whose waves take different rows
constexpr int kMaxParts = 256;                  // of the prefix, and of a request's own keys (the join keeps their weights in LDS)
constexpr int kAll = 0x7FFFFFFF;                // lim0: every row sees every key
constexpr int kRun = 16;                        // keys of a run, see Stream
constexpr float kNone = -3.0e38f;               // running maximum before any key
constexpr float kSlack = 8.f;                   // weights stay below 2^kSlack (kLift higher in fp16)
// Weights are taken against the maximum less kLift.  fp16 has steps of 2^-24 below
// 2^-14: with the largest weight held as 1, those below 2^-25 of it would be lost
// to the value product and still be in l.  Held as 2^7 (2^15 with the slack, fp16
// ends at 2^16), only weights below 2^-32 of it are.  bf16 has fp32's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
constexpr float kWideCap = 64.f;                // caps above it have kernels of their own, see Rows
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How a call is cut into workgroups.  Three kinds of work in one launch:
// prefix (all rows of a key head, the shared keys), few (a request with at most
// kCols rows per key head: the four waves take different keys of each tile and
// are joined at the end; up to kFewTiles such tiles of one request) and many (a
// request with more rows: the waves take different rows).  `joint`: a request's
// workgroups walk the prefix themselves.
struct Plan {
    int pre_tiles, pre_parts, pre_chunk;
    bool pre_few;                    // the rows at the prefix count as few
    int few_parts, few_chunk, few_tiles;
    int many_tiles, many_parts, many_chunk;
    bool joint;
    bool listed;                     // few's units are those that there are, see find_few
    uint32_t pre_units, few_units, many_units;  // (make_plan checks their sum before it narrows them)
    FastDiv by_heads, by_pre_tiles, by_few_parts, by_few_chunk, by_many_tiles;
    int own_parts;                   // partial results of a row from its own keys, at most
    int parts;                       // all partial results of a row; 1: written directly
};

struct KArgs {
    AttnArgs a;
    Plan p;
    float *part_o, *part_m, *part_l;
    int32_t* part_n;
    int G;
    FastDiv per_group;
};

}  // namespace

// ---------------------------------------------------------------------------
// staging
// ---------------------------------------------------------------------------

// LDS tiles of key rows are loaded straight from memory, a row of B bytes after
// the other, with the row's 16-byte chunks c at place c ^ turn(r), so that no
// access meets in a bank: an operand of K is one chunk of 16 rows, a transposing
// load of V takes 4 rows times 64 bytes (8-bit V: 8 rows times 32 bytes).
template <int B>
__device__ __forceinline__ int turn(int r) {  // 16-bit rows
    if constexpr (B == 128) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    else return ((r & 3) << 2) | ((r >> 2) & 3);
}
template <int B>
__device__ __forceinline__ int turn8(int r) {  // 8-bit rows: rows 0-3 and 8-11 (4-7 and 12-15) are read together
    const int b1 = (r >> 1) & 1, b2 = (r >> 2) & 1, b3 = (r >> 3) & 1;
    if constexpr (B == 64) return b2 | (b3 << 1);
    else if constexpr (B == 128) return b2 | (b1 << 1) | (b3 << 2);
    else return b2 | (b1 << 1) | (b3 << 2) | ((r & 1) << 3);
}

// Two floats as 16-bit values in one word, rounded to nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        const v2b p = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, p);
    } else {
        const v2h p = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, p);
    }
}

template <bool BF16>
__device__ __forceinline__ v4u widen8(uint32_t lo, uint32_t hi) {  // 8 E4M3 codes -> 16-bit values (exact)
    v4u o;
    if constexpr (BF16) {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    } else {
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    }
    return o;
}

// u without the elements that are not finite (16-bit: exponent all ones; E4M3:
// the two NaN codes), which become zeros.
template <bool BF16, bool FP8>
__device__ __forceinline__ v4u finite_of(v4u u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        constexpr uint32_t E = FP8 ? 0x7Fu : BF16 ? 0x7F80u : 0x7C00u;
        constexpr int W = FP8 ? 8 : 16;
        uint32_t keep = 0;
#pragma unroll
        for (int b = 0; b < 32; b += W) keep |= (u[i] & (E << b)) == (E << b) ? 0u : (FP8 ? 0xFFu : 0xFFFFu) << b;
        u[i] &= keep;
    }
    return u;
}
__device__ __forceinline__ bool differ(v4u a, v4u b) { return ((a[0] ^ b[0]) | (a[1] ^ b[1]) | (a[2] ^ b[2]) | (a[3] ^ b[3])) != 0; }

// Where key index i of a workgroup is: indices below `shared` are the prefix's,
// the rest are the request's own.
struct Keys {
    const int32_t* pre;
    const int32_t* own;
    int shared;
    __device__ __forceinline__ int32_t page(const KvLayout& kv, int i, uint32_t& at) const {
        const bool s = i < shared;
        const uint32_t j = s ? i : i - shared;
        const uint32_t b = kv.per_block.div(j);
        at = j - b * (uint32_t)kv.block_size;
        return (s ? pre : own)[b];
    }
};

// What a workgroup does.
struct Task {
    Keys keys;
    int kvh, nrows, row0, k0, k1, lim0, part;
    int64_t tok0;
    bool direct;
    // keys below k1 that the rows of token `rtok`, counted from tok0, see
    __device__ __forceinline__ int seen_by(int rtok) const { return min(k1, lim0 == kAll ? k1 : max(keys.shared, lim0 + rtok)); }
};

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ v2u tr16(lds_char* p) { return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)p)); }
__device__ __forceinline__ v2u tr8(lds_char* p) { return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i)p)); }
#endif

// v of lane ^ 32, without a trip through LDS.
__device__ __forceinline__ float other_half(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
    const v2u r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false));
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
#else
    return v;
#endif
}

// Waits for loads into LDS, which the compiler does not follow to their readers:
// until at most N vector loads of this wave are open; until its LDS reads are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <bool BF16>
__device__ __forceinline__ v16f mfma32(const Frag8& a, const Frag8& b, v16f c) {
    if constexpr (BF16) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.b, b.b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_f16(a.h, b.h, c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// one wave's 32 query rows
// ---------------------------------------------------------------------------

// The state of 32 query rows (a wave's matrix columns): lane (col, half) holds
// row col's statistics and its output elements 32 t + 8 (i / 4) + 4 half + i % 4
// (register i of tile t).  Scores come as registers of keys
// kb + 8 (i / 4) + 4 half + i % 4.
template <int DP, bool BF16, bool FP8, bool WIDE>
struct Rows {
    static constexpr int KS = DP / 16, DT = DP / 32;
    Frag8 q[KS];
    v16f acc[DT];
    float m, l;
    float c1, c2, cy, inv;
    bool cap;
    int half, col, lane;
    int seen, wseen;  // keys that this lane's row sees; that every row of the wave sees
    bool live;

    // s = c2 x.k, or with a cap s = c2 tanh(y), y = cy x.k.  tanh_far errs by 2^-22 of
    // the cap: up to kWideCap less than 2^-16 of a weight, far below its rounding.
    // Beyond that it would show, and small y go by the series, whose error is a share
    // of the score: s = c2 (x.k) (tanh(y) / y).  These are kernels of their own (WIDE):
    // 40 requests of drafts and a prompt chunk, cap 30, take 31 us, 38 by the series,
    // and 37 where one kernel holds both ways; prompts without a cap 513 instead of 501.
    __device__ __forceinline__ void init(const KArgs& ka, const Task& w, int wrow0) {
        const AttnArgs& a = ka.a;
        const int D = a.kv.head_dim;
        lane = threadIdx.x & 63;
        half = lane >> 5;
        col = lane & 31;
        const int row = wrow0 + col;
        live = row < w.nrows;
        const int rtok = live ? (int)ka.per_group.div(row) : 0;
        const int64_t tok = w.tok0 + rtok;
        const int head = w.kvh * ka.G + (live ? row - rtok * ka.G : 0);
        seen = w.seen_by(rtok);
        wseen = __builtin_amdgcn_readfirstlane(w.seen_by((int)ka.per_group.div(wrow0 < w.nrows ? wrow0 : 0)));
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = dim_of(s);
            q[s].u = v4u{0u, 0u, 0u, 0u};
            if (live && d < D) q[s].u = ld16((const uint16_t*)a.q + tok * a.q_stride + (int64_t)head * D + d);
        }
        const float ksc = FP8 ? a.k_scale[w.kvh] : 1.f;
        cap = a.softcap > 0.f;
        c2 = (cap && !WIDE ? a.softcap : a.scale * ksc) * kLog2e;
        cy = cap ? fminf(a.scale * ksc / a.softcap, 1e30f) : 0.f;  // (finite: 0 times it is 0)
        c1 = 2.f * kLog2e * cy;
        inv = cap ? a.softcap / (a.scale * ksc) : 0.f;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
        m = kNone;
        l = 0.f;
    }
    // Waits for the query loads here, before the first loads to LDS: the compiler
    // would wait for those too at the first use.
    __device__ __forceinline__ void ready() {
#pragma unroll
        for (int s = 0; s < KS; ++s) asm volatile("" : "+v"(q[s].u));
    }
    // The first of the eight elements that matrix step s takes from this lane:
    // a lane's elements of steps 2g and 2g+1 are neighbours (16 codes of an
    // 8-bit cache are one load).
    __device__ __forceinline__ int dim_of(int s) const { return 32 * (s >> 1) + 16 * half + 8 * (s & 1); }

    // tanh(y) of 2^t = e^2y, to some 2^-22 of 1; and tanh(y) / y of z = y^2 < 1/16, to
    // 2^-22 of itself (the next term is 2^-27).
    __device__ __forceinline__ static float tanh_far(float t) { return 1.f - 2.f * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t)); }
    __device__ __forceinline__ static float tanh_series(float z) {
        return __builtin_fmaf(z, __builtin_fmaf(z, __builtin_fmaf(z, __builtin_fmaf(z, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
    }
    // Scores of keys kb..kb+31: cap and mask, and the running maximum.
    __device__ __forceinline__ void prepare(v16f& st, int kb) {
        // (in the two uniform branches a value passes through an empty asm, so that
        // nothing is computed ahead of the branch)
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y = cy * st[i], z = y * y;
                st[i] = z < 0.0625f ? st[i] * tanh_series(z) : inv * tanh_far(c1 * st[i]);
            }
        } else if (cap) {
            float c = c1;
            asm volatile("" : "+v"(c));
#pragma unroll
            for (int i = 0; i < 16; ++i) st[i] = tanh_far(c * st[i]);
        }
        if (kb + 32 > wseen) {
            int over = seen - kb - 4 * half;
            asm volatile("" : "+v"(over));
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i >> 2) + (i & 3) >= over) st[i] = -INFINITY;
        }
        float mx = st[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, st[i]);
        mx = __builtin_fmaf(fmaxf(mx, other_half(mx)), c2, -kLift<BF16>);
        // The maximum that the weights are taken against only has to keep them in
        // range: it moves, and the sums with it, once it is behind by 2^kSlack.
        if (__any(mx > m + kSlack)) {
            const float to = fmaxf(m, mx), shrink = __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= shrink;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[t][i] *= shrink;
        }
    }
    // Weights of the 32 keys, rounded to 16 bits as the operands of the value
    // product: a relative error of up to 2^-8 (bf16) or 2^-11 (fp16) each, like the
    // output's own, and of up to 2^-32 of the row's largest weight for fp16 weights
    // below 2^-21 of it; their sum is of the unrounded ones.  Weights held in two
    // 16-bit parts would take half as many matrix instructions again.
    __device__ __forceinline__ void weights(const v16f& st, Frag8 (&p)[2]) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(st[8 * k + 2 * j], c2, -m));
                const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(st[8 * k + 2 * j + 1], c2, -m));
                l += x;
                l += y;
                p[k].u[j] = pack2<BF16>(x, y);
            }
    }
    // S^T = K Q^T of 32 keys: rows are keys, columns are queries.
    __device__ __forceinline__ void scores(lds_char* lk, v16f& st) {  // lk: the first of the 32 rows
        constexpr int B = FP8 ? DP : DP * 2;
        typedef const __attribute__((address_space(3))) v4u lds_v4u;
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i] = 0.f;
#pragma unroll
        for (int g = 0; g < DP / 32; ++g) {  // 32 elements: two matrix steps
            Frag8 f0, f1;
            if constexpr (FP8) {
                const v4u u = *(lds_v4u*)(lk + col * B + ((2 * g + half) ^ turn8<B>(col)) * 16);
                f0.u = widen8<BF16>(u[0], u[1]);
                f1.u = widen8<BF16>(u[2], u[3]);
            } else {
                f0.u = *(lds_v4u*)(lk + col * B + ((4 * g + 2 * half) ^ turn<B>(col)) * 16);
                f1.u = *(lds_v4u*)(lk + col * B + ((4 * g + 2 * half + 1) ^ turn<B>(col)) * 16);
            }
            st = mfma32<BF16>(f0, q[2 * g], st);
            st = mfma32<BF16>(f1, q[2 * g + 1], st);
        }
    }
    // O^T += V^T P^T over 32 keys.  A transposing load gives lane (16 dsel + i16,
    // half) element 16 dsel + i16 of four (8-bit: eight) rows, of which each lane
    // names a part: 8 bytes of one row.
    __device__ __forceinline__ void values(lds_char* lv, const Frag8 (&p)[2]) {  // lv: the first of the 32 rows
#if defined(__HIP_DEVICE_COMPILE__)
        const int i16 = lane & 15, dsel = (lane >> 4) & 1;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                Frag8 vf;
                if constexpr (FP8) {
                    const int j = i16 >> 1, r = 16 * k + 4 * half + (j & 3) + 8 * (j >> 2);
                    const v2u a = tr8(lv + r * DP + ((2 * t + dsel) ^ turn8<DP>(r)) * 16 + (i16 & 1) * 8);
                    vf.u = widen8<BF16>(a[0], a[1]);
                } else {
                    const int r = 16 * k + 4 * half + (i16 >> 2), c = 4 * t + 2 * dsel + ((i16 & 3) >> 1);
                    const v2u a = tr16(lv + r * DP * 2 + (c ^ turn<DP * 2>(r)) * 16 + (i16 & 1) * 8);
                    const v2u b = tr16(lv + (r + 8) * DP * 2 + (c ^ turn<DP * 2>(r + 8)) * 16 + (i16 & 1) * 8);
                    vf.u = v4u{a[0], a[1], b[0], b[1]};
                }
                acc[t] = mfma32<BF16>(vf, p[k], acc[t]);
            }
#endif
    }
    // Values that are not finite are left out of the tiles where some row does
    // not see them (0 times infinity would reach that row).  The rows that do
    // see one get it here: its weight is positive, so it can only make the sum
    // that infinity, or NaN.  Keys first..k1-1 of which this wave had those with
    // (key - k0) / 32 % waves == wave.
    __device__ __forceinline__ void add_nonfinite(const KArgs& ka, const Keys& keys, int kvh, int first, int k0, int k1, int waves, int wave) {
        const KvLayout& kv = ka.a.kv;
        for (int key = first; key < k1; ++key) {
            if ((key - k0) / 32 % waves != wave) continue;
            uint32_t at;
            const int32_t b = keys.page(kv, key, at);
            if ((uint32_t)b >= (uint32_t)kv.num_blocks || key >= seen) continue;
            const int64_t off = (int64_t)b * kv.block_stride + (int64_t)at * kv.slot_stride + (int64_t)kvh * kv.head_stride;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int d = 32 * t + 8 * g + 4 * half;
                    if (d >= kv.head_dim) continue;
                    if constexpr (FP8) {
                        const uint32_t w = *(const uint32_t*)((const uint8_t*)ka.a.v_cache + off + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (((w >> (8 * j)) & 0x7Fu) == 0x7Fu) acc[t][4 * g + j] += __builtin_nanf("");
                    } else {
                        const v2u w = *(const v2u*)((const uint16_t*)ka.a.v_cache + off + d);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = bits16_to_f32<BF16>((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
                            if (!(fabsf(v) < INFINITY)) acc[t][4 * g + j] += v;
                        }
                    }
                }
        }
    }
    // The sums of this wave's rows into LDS, as rows of kPitch floats (padded, so
    // that eight rows meet in no bank).
    static constexpr int kPitch = DP + 4;
    __device__ __forceinline__ void spill(lds_float* o) {
        if (!live) return;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *(lds_v4f*)(o + col * kPitch + 32 * t + 8 * g + 4 * half) = v4f{acc[t][4 * g], acc[t][4 * g + 1], acc[t][4 * g + 2], acc[t][4 * g + 3]};
    }
};

// Four elements of a row's result, or of its partial one (m, l and the sum of
// weight times value), to where they belong.  A row that sees no key is 0; one
// that sees keys, whose scores are all minus infinity, has l = 0 too and is NaN.
template <bool BF16, bool FP8>
__device__ __forceinline__ void put(const KArgs& ka, const Task& w, int row, int d, v4f o, float m, float l) {
    const AttnArgs& a = ka.a;
    const int D = a.kv.head_dim, rt = (int)ka.per_group.div(row), head = w.kvh * ka.G + row - rt * ka.G;
    const int64_t tok = w.tok0 + rt, at = tok * a.q_heads + head;
    float f = FP8 ? a.v_scale[w.kvh] : 1.f;
    if (w.direct) {
        if (l == 0.f && w.seen_by(rt) > 0) l = __builtin_nanf("");
        f = l == 0.f ? 0.f : f / l;
        *(uint2*)((uint16_t*)a.out + tok * a.out_stride + (int64_t)head * D + d) = make_uint2(pack2<BF16>(o[0] * f, o[1] * f), pack2<BF16>(o[2] * f, o[3] * f));
        if (d == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    } else {
        *(v4f*)(ka.part_o + ((int64_t)w.part * a.T * a.q_heads + at) * D + d) = o * f;
        if (d == 0) {  // a row's parts side by side
            ka.part_m[at * ka.p.parts + w.part] = m;
            ka.part_l[at * ka.p.parts + w.part] = l;
        }
    }
}

// ---------------------------------------------------------------------------
// keys on their way to LDS
// ---------------------------------------------------------------------------

// Zeros for what is loaded into LDS in place of keys that do not exist.
__device__ __attribute__((aligned(16))) const uint32_t g_zeros[4] = {0, 0, 0, 0};

// 16 bytes a lane from memory to LDS: lane l's go to `to` + 16 l.  The load is
// written out because the compiler, where it sees one, waits for all of them
// before any LDS read or barrier; its readers wait by wait_loads instead.  It has
// no register to return to.
__device__ __forceinline__ void load_to_lds(const char* src, lds_char* to) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((int)__builtin_bit_cast(uint32_t, to))), "v"(src)
                 : "memory", "m0");
#endif
}

// The same from a wave-uniform address and 32-bit offsets of the lanes.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t lane_off, lds_char* to) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((int)__builtin_bit_cast(uint32_t, to))), "v"(lane_off), "s"(base)
                 : "memory", "m0");
#endif
}

// ROWS keys of a wave at a time: place() finds them, fetch() sends their rows to
// LDS.  Pages are counted on from the prefix's first to the request's last; the
// ids of 128 in a row lie in registers, so that a wave asks memory for ids (and
// then waits for all its loads) only once in so many pages.
//
// Where pages hold whole runs of 16 keys (the page size and the prefix are
// multiples of 16) and all keys are there, their addresses are scalar arithmetic
// and an offset that each lane keeps.  Else each lane finds one key, and the
// lanes that load its row get the offset by a shuffle; what is no key, or beyond
// the head, comes from g_zeros.  (Vector instructions are what the tiles of many
// rows have least room for: with the second way alone, 6069 tokens of prompts
// behind 4096 took 607 us instead of 517.)
template <int DP, bool FP8, int ROWS>
struct Stream {
    static constexpr int EB = FP8 ? 1 : 2, B = DP * EB;   // bytes of a row
    static constexpr int LPR = B / 16, RPL = 64 / LPR;    // lanes of a row, rows of a load
    static constexpr int NL = ROWS / RPL, RUNS = ROWS / kRun;
    const KvLayout& kv;
    const Keys& keys;
    const char *k, *v;
    int k1, lane, row_bytes, shared_pages, first = -256;
    uint32_t bstep, sstep;
    bool runs, whole = false;
    int32_t id0 = 0, id1 = 0;  // of pages first + lane, first + 64 + lane
    int64_t off = -1;          // byte offset of this lane's key in the cache, -1 if there is none
    uint64_t run[RUNS];        // of the runs' first keys
    uint32_t in_run[NL];       // this lane's place from there, for each load

    __device__ __forceinline__ Stream(const AttnArgs& a, const Keys& ks, int kvh, int end)
        : kv(a.kv), keys(ks), k((const char*)a.k_cache + (int64_t)kvh * a.kv.head_stride * EB),
          v((const char*)a.v_cache + (int64_t)kvh * a.kv.head_stride * EB), k1(end), lane(threadIdx.x & 63), row_bytes(a.kv.head_dim * EB),
          shared_pages(ks.shared ? (int)a.kv.per_block.div(ks.shared - 1) + 1 : 0), bstep((uint32_t)(a.kv.block_stride * EB)),
          sstep((uint32_t)(a.kv.slot_stride * EB)),
          runs(a.kv.block_size % kRun == 0 && ks.shared % kRun == 0 && row_bytes == B && a.kv.slot_stride < (1 << 26)) {
#pragma unroll
        for (int n = 0; n < NL; ++n) in_run[n] = (uint32_t)(row_of(n) & (kRun - 1)) * sstep + (uint32_t)chunk_of(n) * 16;
    }
    __device__ __forceinline__ int row_of(int n) const { return n * RPL + lane / LPR; }
    __device__ __forceinline__ int chunk_of(int n) const {
        const int r = row_of(n);
        return (lane % LPR) ^ (FP8 ? turn8<B>(r) : turn<B>(r));
    }
    __device__ __forceinline__ int page_of(int i, uint32_t& at) const {
        const bool s = i < keys.shared;
        const uint32_t j = s ? i : i - keys.shared, b = kv.per_block.div(j);
        at = j - b * (uint32_t)kv.block_size;
        return (s ? 0 : shared_pages) + (int)b;
    }
    __device__ __forceinline__ int32_t id_of(int page) const {
        return page < shared_pages ? keys.pre[page] : keys.own[page - shared_pages];
    }
    __device__ __forceinline__ void reach(int lo, int hi) {  // ids of pages lo .. hi (at most 65) into the registers
        if (hi - first >= 128) {
            uint32_t unused;
            const int last = page_of(k1 - 1, unused);
            first = lo;
            id0 = id_of(min(first + lane, last));
            id1 = id_of(min(first + 64 + lane, last));
        }
    }
    __device__ __forceinline__ void place(int kb) {  // keys kb .. kb + ROWS - 1 (kb uniform); there is at least one key before k1
        whole = false;
        if (runs && kb + ROWS <= k1) {
            uint32_t at[RUNS];
            int page[RUNS];
#pragma unroll
            for (int j = 0; j < RUNS; ++j) page[j] = page_of(kb + j * kRun, at[j]);
            reach(page[0], page[RUNS - 1]);
            whole = true;
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                const int p = page[j] - first;
                const uint32_t id = (uint32_t)(p < 64 ? __builtin_amdgcn_readlane(id0, p) : __builtin_amdgcn_readlane(id1, p - 64));
                run[j] = (uint64_t)id * bstep + (uint64_t)at[j] * sstep;
                whole = whole && id < (uint32_t)kv.num_blocks;
            }
            if (whole) return;
        }
        const int i = kb + (lane & (ROWS - 1));
        uint32_t at;
        const int page = page_of(min(i, k1 - 1), at);
        reach(__builtin_amdgcn_readfirstlane(page), __builtin_amdgcn_readlane(page, ROWS - 1));
        const int32_t a = __shfl(id0, page - first), b = __shfl(id1, page - first);  // (modulo 64)
        const uint32_t id = (uint32_t)(page - first < 64 ? a : b);
        off = i < k1 && id < (uint32_t)kv.num_blocks ? (int64_t)((uint64_t)id * bstep + (uint64_t)at * sstep) : (int64_t)-1;
    }
    __device__ __forceinline__ void fetch(const char* base, lds_char* to) {
        if (whole) {
#pragma unroll
            for (int n = 0; n < NL; ++n) load_to_lds(base + run[n * RPL / kRun], in_run[n], to + n * 1024);
        } else {
            const uint32_t lo = (uint32_t)off, hi = (uint32_t)((uint64_t)off >> 32);
#pragma unroll
            for (int n = 0; n < NL; ++n) {
                const int64_t o = (int64_t)(((uint64_t)(uint32_t)__shfl((int)hi, row_of(n)) << 32) | (uint32_t)__shfl((int)lo, row_of(n)));
                load_to_lds(o >= 0 && chunk_of(n) * 16 < row_bytes ? base + o + chunk_of(n) * 16 : (const char*)g_zeros, to + n * 1024);
            }
        }
    }
};

// Takes what is not finite out of `n` kilobytes of a V tile; true if there was any.
template <bool BF16, bool FP8>
__device__ __forceinline__ bool clean(lds_char* lv, int n) {
    bool bad = false;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        auto at = (__attribute__((address_space(3))) v4u*)(lv + i * 1024 + (threadIdx.x & 63) * 16);
        const v4u u = *at, f = finite_of<BF16, FP8>(u);
        bad |= differ(f, u);
        *at = f;
    }
    return bad;
}

// ---------------------------------------------------------------------------
// few rows: a stream of keys per wave
// ---------------------------------------------------------------------------

// Groups of 32 keys that a wave has room for.  16-bit rows fill the LDS of two
// workgroups a CU with one; with half the bytes of an 8-bit cache a second one
// keeps as many bytes on their way.
template <bool FP8>
constexpr int kStages = FP8 ? 2 : 1;

// At most 32 rows.  The cache is read once, so what bounds this is HBM: each
// wave takes every fourth group of 32 keys by itself, with no barrier, into its
// own LDS tiles.  The tile of K is free once the scores are there and the tile of
// V after the value product, and each is asked for again at once, so that nearly
// all the time both are on their way.  64 requests of 4096 keys, 64/8 heads of
// 128: 5.4 TB/s in 16 bits, 4.6 in 8, where a large copy reaches 5.2.  The waves
// are joined at the end.
template <int DP, bool BF16, bool FP8, bool WIDE>
__device__ __forceinline__ void attend_few(const KArgs& ka, const Task& w, lds_char* sk, lds_char* sv) {
    typedef Stream<DP, FP8, 32> S;
    constexpr int NL = S::NL, NS = kStages<FP8>, TILE = 32 * S::B;
    constexpr int STEP = kWaves * 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Rows<DP, BF16, FP8, WIDE> x;
    x.init(ka, w, w.row0);
    S in(ka.a, w.keys, w.kvh, w.k1);
    lds_char* const wk = sk + wave * NS * TILE;  // this wave's tiles
    lds_char* const wv = sv + wave * NS * TILE;
    int kb = w.k0 + wave * 32;
    bool bad = false;
    if (kb < w.k1) in.place(kb);
    x.ready();
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        if (kb + n * STEP < w.k1) {
            if (n) in.place(kb + n * STEP);
            in.fetch(in.k, wk + n * TILE);
            in.fetch(in.v, wv + n * TILE);
        }
    }
    lds_char *lk = wk, *lv = wv;
    for (; kb < w.k1; kb += STEP) {
        const bool next = kb + STEP < w.k1, more = kb + NS * STEP < w.k1;
        // Loads end in order, and K and V of a group are NL each.  After K of this
        // group came its V, and K and V of the groups that are already asked for.
        if (NS == 2 && next) wait_loads<3 * NL>();
        else wait_loads<NL>();
        v16f st;
        x.scores(lk, st);
        if (more) {
            in.place(kb + NS * STEP);
            wait_lds();  // the tile of K has been read
            in.fetch(in.k, lk);
        }
        x.prepare(st, kb);
        Frag8 p[2];
        x.weights(st, p);
        // after V of this group: K and V of the next, K of the one after
        if (more) wait_loads<(2 * NS - 1) * NL>();
        else if (NS == 2 && next) wait_loads<2 * NL>();
        else wait_loads<0>();
        if (min(kb + 32, w.k1) > x.wseen) bad |= clean<BF16, FP8>(lv, NL);  // some row does not see some of these keys
        x.values(lv, p);
        if (more) {
            wait_lds();  // the tile of V has been read
            in.fetch(in.v, lv);
        }
        if constexpr (NS == 2) {
            lk = lk == wk ? wk + TILE : wk;
            lv = lv == wv ? wv + TILE : wv;
        }
    }
    x.l += other_half(x.l);
    if (__any(bad)) x.add_nonfinite(ka, w.keys, w.kvh, x.wseen < w.k0 ? w.k0 : w.k0 + (x.wseen - w.k0) / 32 * 32, w.k0, w.k1, kWaves, wave);

    // The waves' results meet in LDS, and all threads join them, four elements at
    // a time (in a loop, and only the rows there are: with few keys a workgroup's
    // time is the latency of code that it runs once).
    typedef Rows<DP, BF16, FP8, WIDE> R;
    __shared__ float s_m[kWaves][kCols], s_l[kWaves][kCols];
    if (x.half == 0) {
        s_m[wave][x.col] = x.m;
        s_l[wave][x.col] = x.l;
    }
    __syncthreads();
    x.spill((lds_float*)(wave < 2 ? sk : sv) + (wave & 1) * kCols * R::kPitch);
    __syncthreads();
    const int rows = min(kCols, w.nrows - w.row0);
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d >= ka.a.kv.head_dim) continue;
        float m = s_m[0][r], l = 0.f;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) m = fmaxf(m, s_m[v][r]);
        v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const float f = __builtin_amdgcn_exp2f(s_m[v][r] - m);
            l += f * s_l[v][r];
            o += f * *(const lds_v4f*)((lds_float*)(v < 2 ? sk : sv) + ((v & 1) * kCols + r) * R::kPitch + d);
        }
        put<BF16, FP8>(ka, w, w.row0 + r, d, o, m, l);
    }
}

// ---------------------------------------------------------------------------
// many rows: tiles of keys shared by the waves
// ---------------------------------------------------------------------------

// Each wave has 32 rows of its own; tiles of 64 keys are in LDS for all four, in
// two buffers.  What bounds this is the matrix units and, with as many cycles,
// the exponentials, so a wave starts the score product of the next 32 keys before
// it turns the last ones into weights.  A wave fetches 16 rows of each tile; K of
// the tile after the next goes where this tile's was once all have read it, half
// a tile before V does, so each has a whole tile's time to arrive.
template <int DP, bool BF16, bool FP8, bool WIDE>
__device__ __forceinline__ void attend_many(const KArgs& ka, const Task& w, lds_char* sk, lds_char* sv) {
    typedef Stream<DP, FP8, 16> S;
    constexpr int KT = 64, NL = S::NL, TILE = KT * S::B, HALF = 32 * S::B;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wrow0 = w.row0 + wave * kCols;
    const bool wlive = wrow0 < w.nrows;
    Rows<DP, BF16, FP8, WIDE> x;
    x.init(ka, w, wrow0);
    // keys that every row of the workgroup sees
    const int gseen = w.seen_by((int)ka.per_group.div(w.row0));
    S in(ka.a, w.keys, w.kvh, w.k1);
    lds_char* const wk = sk + wave * 16 * S::B;  // this wave's rows of a tile
    lds_char* const wv = sv + wave * 16 * S::B;
    const int mine = wave * 16;
    bool bad = false;
    // Where some row does not see some key, V is cleaned by those that fetched it.
    auto ready_v = [&](int kt, int at) {
        if (min(kt + KT, w.k1) > gseen) {
            bad |= clean<BF16, FP8>(wv + at, NL);
            __syncthreads();
        }
    };
    v16f s0, s1;
    Frag8 p[2];
    if (w.k0 < w.k1) in.place(w.k0 + mine);
    x.ready();
    if (w.k0 < w.k1) {
        in.fetch(in.k, wk);
        in.fetch(in.v, wv);
        in.place(w.k0 + KT + mine);
        in.fetch(in.k, wk + TILE);
        in.fetch(in.v, wv + TILE);
        wait_loads<2 * NL>();  // the first tile is there: the second is younger
        __syncthreads();
        ready_v(w.k0, 0);
        if (wlive) {
            x.scores(sk, s0);
            x.prepare(s0, w.k0);
        }
    }
    // One tile from the buffers at `at`; the next is at `nx`.  On entry: the scores
    // of its first 32 keys.  The last one asks for tiles of nothing but zeros and
    // scores one: with the same steps on every way through, each load is waited for
    // by its place in the queue.
    auto step = [&](int kt, int at, int nx) {
        if (wlive) {
            x.scores(sk + at + HALF, s1);
            x.weights(s0, p);
            x.values(sv + at, p);
            x.prepare(s1, kt + 32);
        }
        wait_loads<NL>();  // K of the next tile: only its V is younger
        __syncthreads();   // and this tile's K has been read
        in.place(kt + 2 * KT + mine);
        in.fetch(in.k, wk + at);
        if (wlive) {
            x.scores(sk + nx, s0);
            x.weights(s1, p);
            x.values(sv + at + HALF, p);
            x.prepare(s0, kt + KT);
        }
        wait_loads<NL>();  // V of the next tile: only the K just asked for is younger
        __syncthreads();   // and this tile's V has been read
        in.fetch(in.v, wv + at);
        if (kt + KT < w.k1) ready_v(kt + KT, nx);
    };
    for (int kt = w.k0; kt < w.k1; kt += 2 * KT) {
        step(kt, 0, TILE);
        if (kt + KT < w.k1) step(kt + KT, TILE, 0);
    }
    wait_loads<0>();  // nothing is on its way to LDS any more
    x.l += other_half(x.l);
    if (__syncthreads_or(bad) && wlive) x.add_nonfinite(ka, w.keys, w.kvh, gseen < w.k0 ? w.k0 : w.k0 + (gseen - w.k0) / KT * KT, w.k0, w.k1, 1, 0);
    // each wave's rows through its own share of the tiles' LDS, so that whole rows are written
    typedef Rows<DP, BF16, FP8, WIDE> R;
    __shared__ float s_m[kWaves][kCols], s_l[kWaves][kCols];
    if (x.half == 0) {
        s_m[wave][x.col] = x.m;
        s_l[wave][x.col] = x.l;
    }
    auto o = (lds_float*)(wave < 2 ? sk : sv) + (wave & 1) * kCols * R::kPitch;
    x.spill(o);
    __syncthreads();
    const int rows = min(kCols, w.nrows - wrow0);
#pragma unroll 4
    for (int i = x.lane; i < rows * (DP / 4); i += 64) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d < ka.a.kv.head_dim) put<BF16, FP8>(ka, w, wrow0 + r, d, *(const lds_v4f*)(o + r * R::kPitch + d), s_m[wave][r], s_l[wave][r]);
    }
}

// A unit of a segment whose workgroups come in groups of `tiles` that read the
// same keys: whole groups go to one XCD (workgroup ids alternate between the 8
// XCDs), so that the group's keys are fetched into one L2 only.
__device__ __forceinline__ bool grouped_unit(uint32_t id, uint32_t groups, FastDiv tiles, uint32_t& group, int& tile) {
    const bool spread = groups % 8 == 0 || groups >= 32;
    const uint32_t j = spread ? id >> 3 : id, g = tiles.div(j);
    tile = (int)(j - g * tiles.d);
    group = spread ? g * 8 + (id & 7) : g;
    return group < groups;
}

__device__ __forceinline__ int first_tile(const int32_t* cu, int r, int G, int T) {
    const int t = min(max(cu[r], 0), T);
    return (int)((int64_t)t * G / kRowsWide) + r;
}
// The request that owns a tile: the last r whose first tile is not beyond it.
// The lanes of a wave look at 64 requests at a time.
__device__ __forceinline__ int find_request(const int32_t* cu, int B, int tile, int G, int T) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = B;  // among requests lo .. lo + n - 1, lo's first tile is not beyond
    while (n > 1) {
        const int step = (n + 63) / 64, r = lo + lane * step;
        const uint64_t hit = __ballot(lane * step < n && first_tile(cu, r < B ? r : B - 1, G, T) <= tile);
        const int k = hit ? 63 - __builtin_clzll(hit) : 0;
        n = min(step, n - k * step);
        lo += k * step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The `unit`-th of the parts (and tiles) that the requests with few rows have,
// from their lengths: a lane counts one request's, and a running sum says whose
// it is.  False if there are fewer.
__device__ __forceinline__ bool find_few(const KArgs& ka, int unit, int& r, int& part, int& tile) {
    const AttnArgs& a = ka.a;
    const int lane = threadIdx.x & 63, B = (int)a.B, shared = ka.p.joint ? (int)a.prefix_len : 0;
    for (int b0 = 0; b0 < B; b0 += 64) {
        int units = 0, tiles = 1;
        if (b0 + lane < B) {
            const int i = b0 + lane, t0 = max(a.cu[i], 0), fresh = (int)min((int64_t)a.cu[i + 1], a.T) - t0;
            const int64_t rows = min((int64_t)max(fresh, 0), a.max_new) * ka.G;
            if (rows > 0 && rows <= kFewTiles * kCols) {
                const int64_t len = min(max((int64_t)a.kv_lens[i], (int64_t)0), (int64_t)1 << 29);
                const int held = shared + (int)min(min(len, a.max_kv), a.max_blocks * a.kv.block_size);
                const int end = min(held, max(shared, shared + (int)len - fresh + 1 + (int)ka.per_group.div((int)rows - 1)));
                tiles = rows > kCols ? kFewTiles : 1;
                units = max((int)ka.p.by_few_chunk.div(end + ka.p.few_chunk - 1), 1) * tiles;
            }
        }
        int sum = units;
        for (int o = 1; o < 64; o *= 2) {
            const int v = __shfl_up(sum, o);
            if (lane >= o) sum += v;
        }
        const uint64_t hit = __ballot(sum > unit);
        if (hit) {
            const int l = __builtin_ctzll(hit), n = __builtin_amdgcn_readlane(tiles, l);
            const int at = unit - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(units, l));
            r = b0 + l;
            part = n > 1 ? at / kFewTiles : at;
            tile = at - part * n;
            return true;
        }
        unit -= __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

template <int DP, bool BF16, bool FP8, bool WIDE>
__global__ __launch_bounds__(kThreads, DP == 256 ? 1 : 2) void attn_kernel(KArgs ka) {
    // two tiles of 64 rows of K and of V, or the four waves' tiles of 32 (8 bits:
    // twice two); then the results of two waves in each
    constexpr int kTiles = 2 * 64 * DP * 2, kResults = 2 * kCols * Rows<DP, BF16, FP8, WIDE>::kPitch * 4;
    __shared__ __attribute__((aligned(16))) char s_k[kTiles > kResults ? kTiles : kResults], s_v[kTiles > kResults ? kTiles : kResults];
    const AttnArgs& a = ka.a;
    const Plan& p = ka.p;
    uint32_t id = blockIdx.x;
    const bool direct = p.parts == 1;
    const uint32_t heads = a.kv.kv_heads;
    bool few;
    int kvh, part, base, row0, rows, k1, lim0;
    int64_t tok0, k0;
    Keys keys{a.prefix_table, nullptr, (int)a.prefix_len};
    if (id < p.pre_units) {
        uint32_t group;
        int tile;
        if (!grouped_unit(id, heads * p.pre_parts, p.by_pre_tiles, group, tile)) return;
        few = p.pre_few;
        part = (int)p.by_heads.div(group);
        kvh = (int)(group - part * heads);
        base = 0;
        row0 = tile * (few ? kCols : kRowsWide);
        rows = (int)a.T * ka.G;
        tok0 = 0;
        k0 = (int64_t)part * p.pre_chunk;
        k1 = (int)min(k0 + p.pre_chunk, a.prefix_len);
        lim0 = kAll;
    } else {
        id -= p.pre_units;
        few = id < p.few_units;
        int r, tile = 0;
        if (few) {  // heads side by side: together they read whole pages
            uint32_t g = p.by_heads.div(id);
            kvh = (int)(id - g * heads);
            if (p.listed) {
                if (!find_few(ka, (int)g, r, part, tile)) return;
            } else {
                if (p.few_tiles > 1) {
                    tile = g % kFewTiles;
                    g /= kFewTiles;
                }
                r = (int)p.by_few_parts.div(g);
                part = (int)(g - r * p.few_parts);
            }
        } else {
            uint32_t group;
            if (!grouped_unit(id - p.few_units, heads * p.many_parts, p.by_many_tiles, group, tile)) return;
            part = (int)p.by_heads.div(group);
            kvh = (int)(group - part * heads);
            // The last tiles see the most keys: first.  Request r's tiles begin at
            // floor(cu[r] G / kRowsWide) + r, which leaves each at least what it needs.
            tile = p.many_tiles - 1 - tile;
            r = find_request(a.cu, (int)a.B, tile, ka.G, (int)a.T);
            tile -= first_tile(a.cu, r, ka.G, (int)a.T);
        }
        int64_t t0 = a.cu[r], t1 = a.cu[r + 1];
        t0 = t0 < 0 ? 0 : t0;
        t1 = t1 > a.T ? a.T : t1;
        const int fresh = t1 > t0 ? (int)(t1 - t0) : 0;
        tok0 = t0;
        rows = (int)min((int64_t)fresh, a.max_new) * ka.G;
        row0 = tile * (few ? kCols : kRowsWide);
        if (few != (rows <= kFewTiles * kCols) || row0 >= rows) return;
        const int64_t len = min(max((int64_t)a.kv_lens[r], (int64_t)0), (int64_t)1 << 29);
        keys.own = a.block_table + (int64_t)r * a.max_blocks;
        keys.shared = p.joint ? (int)a.prefix_len : 0;
        lim0 = keys.shared + (int)len - fresh + 1;
        const int held = keys.shared + (int)min(min(len, a.max_kv), a.max_blocks * a.kv.block_size);  // keys that can be read
        const int chunk = few ? p.few_chunk : p.many_chunk;
        const int last = min(row0 + (few ? kCols : kRowsWide), rows) - 1;
        const int end = min(held, max(keys.shared, lim0 + (int)ka.per_group.div(last)));  // keys that the tile's last row sees
        k0 = (int64_t)part * chunk;
        base = p.pre_parts;
        // how many parts each token's own keys have, for the join
        if (!direct && part == 0 && kvh == 0)
            for (int i = threadIdx.x; i <= last - row0; i += kThreads) {
                const int t = (int)ka.per_group.div(row0 + i);
                ka.part_n[t0 + t] = (min(held, max(keys.shared, lim0 + t)) + chunk - 1) / chunk;
            }
        if (k0 >= end && !(direct && part == 0)) return;
        k1 = (int)min(k0 + chunk, (int64_t)end);
    }
    const Task w{keys, kvh, rows, row0, (int)k0, k1, lim0, base + part, tok0, direct};
    if (few) attend_few<DP, BF16, FP8, WIDE>(ka, w, (lds_char*)s_k, (lds_char*)s_v);
    else attend_many<DP, BF16, FP8, WIDE>(ka, w, (lds_char*)s_k, (lds_char*)s_v);
}

// Joins the parts of every row.  A workgroup takes `rpw` rows; the weights of
// their parts come first, into LDS, and then D / 4 threads a row add four
// elements each, `spl` times side by side over every spl-th part.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(KArgs ka, int rpw, int spl) {
    extern __shared__ __attribute__((aligned(16))) float s_w[];  // [rpw][parts] weights, then [spl][rpw][D] sums
    __shared__ float s_l[kThreads], s_m[kThreads];
    const AttnArgs& a = ka.a;
    const int D = a.kv.head_dim, parts = ka.p.parts, tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * rpw, rows = a.T * a.q_heads, end = a.cu[a.B];
    auto parts_of = [&](int64_t row) {
        const int64_t tok = row / a.q_heads;
        if (row >= rows || tok >= end) return 0;
        const int own = ka.part_n[tok];
        return ka.p.pre_parts + (own < 0 ? 0 : own > ka.p.own_parts ? ka.p.own_parts : own);
    };
    {
        // lanes 0 .. g-1 of a group of g threads: one row's parts
        const int g = kThreads / rpw < 64 ? kThreads / rpw : 64;
        const int sub = tid / g, i0 = tid % g;
        const int64_t row = row0 + sub;
        const int n = sub < rpw ? parts_of(row) : 0;
        float m = kNone, l = 0.f;
        for (int p = i0; p < n; p += g) m = fmaxf(m, ka.part_m[row * parts + p]);
        for (int o = g / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
        for (int p = i0; p < n; p += g) {
            const float f = __builtin_amdgcn_exp2f(ka.part_m[row * parts + p] - m);
            s_w[sub * parts + p] = f;
            l += f * ka.part_l[row * parts + p];
        }
        for (int o = g / 2; o; o >>= 1) l += __shfl_xor(l, o);
        if (i0 == 0 && sub < rpw) {
            s_m[sub] = m;
            s_l[sub] = l;
        }
    }
    __syncthreads();
    const int tpr = D / 4, d4 = tid % tpr, sub = tid / tpr % rpw, s = tid / tpr / rpw;
    const int64_t row = row0 + sub;
    const int n = s < spl ? parts_of(row) : 0;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    const float* src = ka.part_o + row * D + 4 * d4;
    const int64_t step = rows * D;
#pragma unroll 8
    for (int p = s; p < n; p += spl) {
        const v4f x = *(const v4f*)(src + p * step);
        const float f = s_w[sub * parts + p];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += f * x[j];
    }
    if (spl > 1) {
        __syncthreads();
        if (s < spl) *(v4f*)(s_w + ((s * rpw + sub) * tpr + d4) * 4) = o;
        __syncthreads();
        if (s) return;
        for (int k = 1; k < spl; ++k) o += *(const v4f*)(s_w + ((k * rpw + sub) * tpr + d4) * 4);
    }
    const int64_t tok = row / a.q_heads, hd = row - tok * a.q_heads;
    if (s || row >= rows || tok >= end) return;
    float l = s_l[sub];
    if (l == 0.f && n > 0) l = __builtin_nanf("");  // it sees keys: see put
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *(uint2*)((uint16_t*)a.out + tok * a.out_stride + hd * D + 4 * d4) = make_uint2(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv));
    if (a.lse && d4 == 0) a.lse[row] = l == 0.f ? -INFINITY : (s_m[sub] + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static int pad_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

static int64_t group_units(int64_t groups, int64_t tiles) {  // grouped_unit's ids
    return (groups % 8 == 0 || groups >= 32 ? cdiv(groups, 8) * 8 : groups) * tiles;
}

// Returns the number of workgroups, or -1 if a launch does not hold them.
static int64_t make_plan(const AttnArgs& a, Plan& p) {
    p = Plan{};
    const int64_t hk = a.kv.kv_heads, G = a.q_heads / hk, P = a.prefix_len;
    const int64_t rows = a.T * G;
    const int64_t slots = pad_dim(a.kv.head_dim) == 256 ? 256 : 512;  // workgroups that run at once
    const int64_t total = a.total_kv > 0 ? a.total_kv : a.B * a.max_kv;
    const int64_t bytes = a.kv.dtype == HQ_DT_FP8_E4M3 ? 1 : 2;
    const bool many = a.max_new * G > kFewTiles * kCols;
    const int64_t own_tiles = many ? cdiv(rows, kRowsWide) + a.B : a.B;
    // Own keys of a workgroup.  The lengths are only known on the card (where their
    // sum is not given, every request counts with the bound of its length), so chunks
    // are equal, and two a slot rather than one even out requests of different
    // lengths (17 requests of 4k to 32k keys, 8 heads, E4M3: one 130 us, two 111,
    // four 129).  Where that gives 512 keys or fewer, a workgroup's time is latency.
    // If those of 256 keys take half the slots at most: one part up to 640 keys, for
    // a join costs as much as some 400 (8 requests of 600 keys, 32/8 heads: one part
    // 11.5 us, two 13.4, three 12.6), else 256 a workgroup (900 keys: 13.3 us, with
    // 512 a workgroup 15.3; 700 keys of 256, 16/1 heads: 17.6, in two parts 19.6, in
    // one 20.7).  With more workgroups, one part up to 768 (64 requests of 700 keys:
    // 31 us, in two 38), else 512 (8 of 4000: 28.6, with 256 32).
    auto chunk_of = [&](int64_t extra) {
        const int64_t own = total + extra * a.B, longest = a.max_kv + extra;
        const int64_t work = hk * (many ? own / a.B * own_tiles : own);
        int64_t room = slots * 2 - (many ? 0 : hk * a.B / 2);
        if (room < slots / 2) room = slots / 2;
        const int64_t per = cdiv(cdiv(work, room), 128) * 128;
        if (per > 512) return per;
        const bool small = work <= slots / 2 * 256;
        if (longest <= (small ? 640 : 768)) return (int64_t)768;
        return small && !many && P == extra ? (int64_t)256 : (int64_t)512;
    };
    // A request's workgroups walk the prefix themselves if there is nobody to share
    // it with; if its rows fill 16 tiles, where a product for all gains nothing and
    // parts to join cost (4 prompts of 1517 tokens behind 4096: 550 us, shared 637;
    // 8 of 200 behind 2000: 116, shared 101); and if then no join is left and what
    // could have been shared takes less time than it, about 128 MB out of the L2s
    // (32/8 heads, 64 requests of 100 keys behind 400, 103 MB: 13.8 us, shared 20.6;
    // 256 of 200 behind 128, 134 MB: 45.7, 48.4; behind 256, 267 MB: 50.6, 48.6).
    if (P > 0)
        p.joint = a.B == 1 || rows >= a.B * 16 * kRowsWide ||
                  (P + a.max_kv <= chunk_of(P) && P * (a.B - 1) * hk <= ((int64_t)128 << 20) / (a.kv.head_dim * 2 * bytes));
    const int64_t extra = p.joint ? P : 0, pre_keys = p.joint ? 0 : P;
    const int64_t longest = a.max_kv + extra > 0 ? a.max_kv + extra : 1, per = chunk_of(extra);
    auto split = [&](int64_t keys, int64_t per, int64_t step, int& chunk, int& parts) {  // equal chunks of about `per` keys
        int64_t n = cdiv(keys, per);
        if (n > kMaxParts) n = kMaxParts;
        chunk = (int)(cdiv(cdiv(keys, n), step) * step);
        parts = (int)cdiv(keys, chunk);
    };
    int64_t pre_units = 0, many_units = 0;
    bool whole = false;
    if (many) {
        // Tiles of 128 rows take 64 keys in 2 us or more, so n parts take 35 ns for
        // each of the longest request's keys / n, or for the slots' share of all keys
        // if that is more; a part of all rows is written and read at some 2.5 TB/s,
        // and a join takes 8 us where there would be none (2 requests of 256 tokens at
        // 6000 keys, 32/8 heads: 78 us in 4 parts, 91 in 7; 3 prompts of some 440 up to
        // 1048 keys, 40/8, E4M3: 55 in one, 73 in 3; 4 of 64 at 700: 29 in one, 32 in 4).
        // Every tile counts with the average length of all requests, and where one part
        // is best here, the few rows of the others have one too, which leaves them no
        // join.  Both hold where the others' keys are not many more: long decodes beside
        // a chunk of a prompt are not cut (a chunk of 8192 tokens 599 us, a decode of
        // 131072 keys, 32/8 heads of 128, 113; in one call 1529).
        int64_t best = 0, n = 1;
        const int64_t key = pad_dim(a.kv.head_dim) == 256 ? 70 : 35, avg = total / a.B + extra;
        const int64_t share = hk * avg * (rows / kRowsWide + cdiv(a.B, 2)) / slots;
        const int64_t part = a.T * a.q_heads * a.kv.head_dim * 8 / 2500 * avg / longest;  // of the requests that have it
        for (int64_t i = 1; i <= 64 && i <= cdiv(longest, 128); ++i) {
            const int64_t keys = cdiv(longest, i), join = i > 1 && !pre_keys ? 8000 : 0;
            const int64_t ns = key * (keys > share ? keys : share) + (i > 1 || pre_keys ? i * part : 0) + join;
            if (i == 1 || ns < best) best = ns, n = i;
        }
        split(longest, cdiv(longest, n), 64, p.many_chunk, p.many_parts);
        whole = n == 1 && !pre_keys;
        p.many_tiles = (int)(rows / kRowsWide + a.B);
        many_units = group_units(hk * p.many_parts, p.many_tiles);
    }
    split(longest, whole ? longest : per, 128, p.few_chunk, p.few_parts);
    p.few_tiles = a.max_new * G > kCols ? kFewTiles : 1;
    // Most of requests x parts may be none: workgroups that find no work end at some
    // 350 a us, so with a quarter of them or more the units are listed from the
    // lengths (one request for a lane; the sum of the lengths bounds their number; 17
    // requests of 4k to 32k keys, E4M3: 107 us without the list, 101 with; 73 of up to
    // 5843, half of them without a new token: 30, 25).
    int64_t few_units = a.B * p.few_parts;
    const int64_t there = (total + extra * a.B) / p.few_chunk + a.B;
    p.listed = a.B <= 512 && there * 4 <= few_units * 3;
    if (p.listed) few_units = there;
    few_units *= hk * p.few_tiles;
    if (pre_keys) {
        p.pre_few = rows <= kFewTiles * kCols;
        p.pre_tiles = (int)cdiv(rows, p.pre_few ? kCols : kRowsWide);
        // The prefix's workgroups (bound by the matrix units) run beside those of the
        // own keys (bound by memory), in half the slots: one a CU.  A workgroup for
        // every slot writes and joins twice the parts (64 requests of 500 keys behind
        // 16384, 32/8 heads: 53 us, 66 so, 62 with a quarter of the slots).
        const int64_t work = hk * pre_keys * p.pre_tiles;
        int64_t own_units = there < a.B * p.few_parts ? there : a.B * p.few_parts;
        if (many) own_units = (rows / kRowsWide + cdiv(a.B, 2)) * cdiv(total / a.B + 1, p.many_chunk);
        own_units *= hk;
        int64_t pp = cdiv(work, slots / 2);
        if (pp < 512) {
            // Fewer than 512 keys in the slots that the own keys leave, a quarter at
            // least, where those do not take longer anyhow and a part of all rows is
            // little to write and read (24 requests of 300 keys behind 1000, 32/8 heads:
            // 31 us in 2 parts, 21 in 8; 64 behind 2000: 33 in 4, 31 in 8, 34 in 16; 17
            // of 4k to 32k behind 2011, E4M3: 107 in 4, 111 in 8).  With few rows 128
            // keys are one turn: 384 at least (8 requests of 300 behind 2000: 15.7 us
            // with 512, 14.5 with 384, 15.5 with 128).
            int64_t room = slots - own_units, least = p.pre_few ? 384 : 128;
            room = room > slots / 2 ? slots / 2 : room < slots / 4 ? slots / 4 : room;
            if (own_units > slots * 2 || a.T * a.q_heads * a.kv.head_dim * 8 > (int64_t)8 << 20) least = 512;
            pp = cdiv(work, room);
            pp = pp < least ? least : pp > 512 ? 512 : pp;
        }
        split(pre_keys, cdiv(pp, 64) * 64, 64, p.pre_chunk, p.pre_parts);
        pre_units = group_units(hk * p.pre_parts, p.pre_tiles);
    }
    p.own_parts = p.few_parts > p.many_parts ? p.few_parts : p.many_parts;
    p.parts = p.pre_parts + p.own_parts;
    const int64_t units = pre_units + few_units + many_units;
    // fewer than 2^32 threads in a launch; the join has 4 rows a workgroup or more when there are many
    if (units >= (int64_t)1 << 24 || (p.parts > 1 && cdiv(a.T * a.q_heads, 4) >= (int64_t)1 << 24)) return -1;
    p.pre_units = (uint32_t)pre_units;
    p.few_units = (uint32_t)few_units;
    p.many_units = (uint32_t)many_units;
    p.by_heads = FastDiv::of((uint32_t)hk);
    p.by_few_chunk = FastDiv::of((uint32_t)p.few_chunk);
    p.by_few_parts = FastDiv::of((uint32_t)p.few_parts);
    if (p.pre_tiles) p.by_pre_tiles = FastDiv::of((uint32_t)p.pre_tiles);
    if (many) p.by_many_tiles = FastDiv::of((uint32_t)p.many_tiles);
    return units;
}

static size_t up256(size_t b) { return (b + 255) / 256 * 256; }

size_t attn_workspace(const AttnArgs& a) {
    Plan p;
    if (make_plan(a, p) < 0) return SIZE_MAX;
    if (p.parts == 1) return 0;
    const size_t rows = (size_t)a.T * a.q_heads;
    return up256((size_t)p.parts * rows * a.kv.head_dim * 4) + 2 * up256((size_t)p.parts * rows * 4) + up256((size_t)a.T * 4);
}

template <int DP, bool BF16, bool FP8>
static hipError_t launch_one(const KArgs& ka, int64_t units) {
    const bool wide = ka.a.softcap > kWideCap;
    if (plan_recorder()) {
        plan_record("attn<%d,%s,%s%s> grid=%lld prefix=%d few=%d many=%d joint=%d listed=%d", DP, BF16 ? "bf16" : "fp16", FP8 ? "e4m3" : "16",
                    wide ? ",wide" : "", (long long)units, ka.p.pre_parts, ka.p.few_parts, ka.p.many_parts, (int)ka.p.joint, (int)ka.p.listed);
        return hipSuccess;
    }
    if (wide) hipLaunchKernelGGL((attn_kernel<DP, BF16, FP8, true>), dim3((unsigned)units), dim3(kThreads), 0, ka.a.stream, ka);
    else hipLaunchKernelGGL((attn_kernel<DP, BF16, FP8, false>), dim3((unsigned)units), dim3(kThreads), 0, ka.a.stream, ka);
    return hipGetLastError();
}

template <int DP>
static hipError_t launch_dim(const KArgs& ka, int64_t units) {
    const bool fp8 = ka.a.kv.dtype == HQ_DT_FP8_E4M3;
    if (ka.a.bf16) return fp8 ? launch_one<DP, true, true>(ka, units) : launch_one<DP, true, false>(ka, units);
    return fp8 ? launch_one<DP, false, true>(ka, units) : launch_one<DP, false, false>(ka, units);
}

hipError_t attn_launch(const AttnArgs& a) {
    KArgs ka{};
    ka.a = a;
    const int64_t units = make_plan(a, ka.p);
    if (units < 1) return hipErrorInvalidConfiguration;
    ka.G = a.q_heads / a.kv.kv_heads;
    ka.per_group = FastDiv::of((uint32_t)ka.G);
    if (ka.p.parts > 1 && !plan_recorder()) {  // (a plan has no workspace to lay out)
        const size_t rows = (size_t)a.T * a.q_heads;
        char* w = (char*)a.ws;
        ka.part_o = (float*)w;
        w += up256((size_t)ka.p.parts * rows * a.kv.head_dim * 4);
        ka.part_m = (float*)w;
        w += up256((size_t)ka.p.parts * rows * 4);
        ka.part_l = (float*)w;
        w += up256((size_t)ka.p.parts * rows * 4);
        ka.part_n = (int32_t*)w;
    }
    const int dp = pad_dim(a.kv.head_dim);
    hipError_t e = dp == 64 ? launch_dim<64>(ka, units) : dp == 128 ? launch_dim<128>(ka, units) : launch_dim<256>(ka, units);
    if (e != hipSuccess || ka.p.parts == 1) return e;
    // As many rows a workgroup as its threads hold; with fewer rows than fill the
    // card so, fewer rows and the parts side by side.
    const int fit = kThreads / (a.kv.head_dim / 4);
    const int64_t rows = a.T * a.q_heads;
    int rpw = 1;
    while (rpw * 2 <= fit && rpw < 16 && rows / (rpw * 2) >= 512) rpw *= 2;
    int spl = fit / rpw;
    if (spl > ka.p.parts) spl = ka.p.parts;
    const int64_t wgs = cdiv(rows, rpw);
    size_t shared = (size_t)rpw * ka.p.parts * 4;
    if (shared < (size_t)spl * rpw * a.kv.head_dim * 4) shared = (size_t)spl * rpw * a.kv.head_dim * 4;
    if (plan_recorder()) {
        plan_record("attn_join<%s> grid=%lld parts=%d", a.bf16 ? "bf16" : "fp16", (long long)wgs, ka.p.parts);
        return hipSuccess;
    }
    if (a.bf16) hipLaunchKernelGGL((attn_join_kernel<true>), dim3((unsigned)wgs), dim3(kThreads), shared, ka.a.stream, ka, rpw, spl);
    else hipLaunchKernelGGL((attn_join_kernel<false>), dim3((unsigned)wgs), dim3(kThreads), shared, ka.a.stream, ka, rpw, spl);
    return hipGetLastError();
}

}  // namespace hq
