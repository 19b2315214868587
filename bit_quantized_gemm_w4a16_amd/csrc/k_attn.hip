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

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 32;                       // query rows of a wave's matrix tile
constexpr int kRowsWide = kWaves * kCols;       // rows of a workgroup whose waves take different rows
constexpr int kAll = 0x7FFFFFFF;               // lim0: every row sees every key
constexpr float kNone = -3.0e38f;               // running maximum before any key
constexpr float kSlack = 8.f;                   // weights stay below 2^kSlack
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How a call is cut into workgroups.  Three kinds of work in one launch:
// prefix (all rows of a key head, the shared keys), few (a request with at most
// kCols rows per key head: the four waves take different keys of each tile and
// are joined at the end) and many (a request with more rows: the waves take
// different rows).  `joint`: a request's workgroups walk the prefix themselves.
struct Plan {
    int pre_tiles, pre_parts, pre_chunk;
    bool pre_few;                    // the prefix rows fit one wave's tile
    int few_parts, few_chunk;
    int many_tiles, many_parts, many_chunk;
    bool joint;
    int64_t pre_units, few_units, many_units;
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

// LDS tiles of the key rows, where loads of all 64 banks at once must not meet:
// an operand of K is one 16-byte chunk of 16 rows, a transposing load of V takes
// 4 rows times 64 bytes (8-bit V: 8 rows times 32 bytes).
//
// Tiles that go through registers (many rows) have padded rows, K by 16 bytes
// and V to 64 modulo 256, so that every operand is one address and a constant.
template <int DP>
struct Padded {
    static constexpr int K = DP * 2 + 16, V = DP * 2 + 64;
};
// Tiles that are loaded straight into LDS (few rows) are dense, a row of B bytes
// after the other, and instead the row's 16-byte chunks c change places: c ^
// turn(r), with the same pairs of chunks staying neighbours.
template <int B>
__device__ __forceinline__ int turn(int r) {  // 16-bit rows
    if constexpr (B == 128) return (((r >> 1) & 1) << 2) | (((r >> 2) & 1) << 1);
    else return ((r & 3) << 2) | (((r >> 2) & 1) << 1);
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

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ v2u tr16(lds_char* p) { return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)p)); }
__device__ __forceinline__ v2u tr8(lds_char* p) { return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i)p)); }
#endif

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
template <int DP, bool BF16, bool FP8>
struct Rows {
    static constexpr int KS = DP / 16, DT = DP / 32;
    Frag8 q[KS];
    v16f acc[DT];
    float m, l;
    float c1, c2;
    bool cap;
    int half, col, lane;
    int64_t tok;
    int head, seen, wseen;  // keys that this lane's row sees; that every row of the wave sees
    bool live;

    // s = c2 x.k, or with a cap s = c2 tanh(y), tanh(y) = 1 - 2 / (1 + 2^(c1 x.k))
    __device__ __forceinline__ void init(const KArgs& ka, const Keys& keys, int kvh, int64_t tok0, int nrows, int wrow0, int k1, int lim0) {
        const AttnArgs& a = ka.a;
        const int D = a.kv.head_dim;
        lane = threadIdx.x & 63;
        half = lane >> 5;
        col = lane & 31;
        const int row = wrow0 + col;
        live = row < nrows;
        const int rtok = live ? (int)ka.per_group.div(row) : 0;
        tok = tok0 + rtok;
        head = kvh * ka.G + (live ? row - rtok * ka.G : 0);
        const int wtok = (int)ka.per_group.div(wrow0 < nrows ? wrow0 : 0);
        seen = min(k1, lim0 == kAll ? k1 : max(keys.shared, lim0 + rtok));
        wseen = __builtin_amdgcn_readfirstlane(min(k1, lim0 == kAll ? k1 : max(keys.shared, lim0 + wtok)));
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = dim_of(s);
            q[s].u = v4u{0u, 0u, 0u, 0u};
            if (live && d < D) q[s].u = ld16((const uint16_t*)a.q + tok * a.q_stride + (int64_t)head * D + d);
        }
        const float ksc = FP8 ? a.k_scale[kvh] : 1.f;
        cap = a.softcap > 0.f;
        c1 = cap ? 2.f * kLog2e * a.scale * ksc / a.softcap : 0.f;
        c2 = cap ? a.softcap * kLog2e : a.scale * ksc * kLog2e;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
        m = kNone;
        l = 0.f;
    }
    // Waits for the query loads here: were they still open on some way into a
    // loop, every first use in it would wait for all loads in flight.
    __device__ __forceinline__ void ready() {
#pragma unroll
        for (int s = 0; s < KS; ++s) asm volatile("" : "+v"(q[s].u));
    }
    // The first of the eight elements that matrix step s takes from this lane:
    // a lane's elements of steps 2g and 2g+1 are neighbours (16 codes of an
    // 8-bit cache are one load).
    __device__ __forceinline__ int dim_of(int s) const { return 32 * (s >> 1) + 16 * half + 8 * (s & 1); }

    // Scores of keys kb..kb+31: cap and mask, and the running maximum.
    __device__ __forceinline__ void prepare(v16f& st, int kb) {
        // (in the two uniform branches a value passes through an empty asm, so that
        // nothing is computed ahead of the branch)
        if (cap) {
            float c = c1;
            asm volatile("" : "+v"(c));
#pragma unroll
            for (int i = 0; i < 16; ++i)
                st[i] = 1.f - 2.f * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(c * st[i]));
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
        mx = fmaxf(mx, __shfl_xor(mx, 32)) * c2;
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
    // product (relative error 2^-9 or 2^-12 each, like the output's own rounding);
    // their sum is of the unrounded ones.
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
    // O^T += V^T P^T over 32 keys.  A transposing load gives lane (16 dsel + i16,
    // half) element 16 dsel + i16 of four (8-bit: eight) rows, of which each lane
    // names a part: 8 bytes of one row.
    __device__ __forceinline__ void values_padded(lds_char* lv, const Frag8 (&p)[2]) {  // lv: the first of the 32 rows
#if defined(__HIP_DEVICE_COMPILE__)
        const int i16 = lane & 15, dsel = (lane >> 4) & 1;
        lds_char* v = lv + (4 * half + (i16 >> 2)) * Padded<DP>::V + 32 * dsel + 8 * (i16 & 3);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int t = 0; t < DT; ++t) {
                const v2u a = tr16(v + 16 * k * Padded<DP>::V + 64 * t), b = tr16(v + (16 * k + 8) * Padded<DP>::V + 64 * t);
                Frag8 vf;
                vf.u = v4u{a[0], a[1], b[0], b[1]};
                acc[t] = mfma32<BF16>(vf, p[k], acc[t]);
            }
#endif
    }
    __device__ __forceinline__ void values_dense(lds_char* lv, const Frag8 (&p)[2]) {
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
    // The rows' result, or their partial one: (m, l, sum of weight times value).
    __device__ __forceinline__ void store(const KArgs& ka, int kvh, int part, bool direct) {
        const AttnArgs& a = ka.a;
        const int D = a.kv.head_dim;
        if (!live) return;
        const float vsc = FP8 ? a.v_scale[kvh] : 1.f;
        const int64_t pr = ((int64_t)part * a.T + tok) * a.q_heads + head;
        const float f = !direct ? vsc : l > 0.f || l != l ? vsc / l : 0.f;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int d = 32 * t + 8 * g + 4 * half;
                if (d >= D) continue;
                v4f o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = acc[t][4 * g + j] * f;
                if (direct)
                    *(uint2*)((uint16_t*)a.out + tok * a.out_stride + (int64_t)head * D + d) = make_uint2(pack2<BF16>(o[0], o[1]), pack2<BF16>(o[2], o[3]));
                else
                    *(v4f*)(ka.part_o + pr * D + d) = o;
            }
        if (half == 0) {
            if (!direct) {
                ka.part_m[pr] = m;
                ka.part_l[pr] = l;
            } else if (a.lse) {
                a.lse[tok * a.q_heads + head] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
            }
        }
    }
};

// What a workgroup does.
struct Task {
    Keys keys;
    int kvh, nrows, row0, k0, k1, lim0, part;
    int64_t tok0;
    bool direct;
};

// ---------------------------------------------------------------------------
// few rows: a stream of keys per wave
// ---------------------------------------------------------------------------

// Zeros for what is loaded into LDS in place of keys that do not exist.
__device__ __attribute__((aligned(16))) const uint32_t g_zeros[4] = {0, 0, 0, 0};

// At most 32 rows.  The cache is read once, so what bounds this is HBM: each
// wave takes every fourth group of 32 keys by itself, with no barrier, straight
// from memory into its own LDS tiles.  The tile of K is free once the scores are
// there and the tile of V after the value product, and each is asked for again
// at once, so that nearly all the time both are on their way.  A lane looks up
// the page of one key; the lanes that load that key's row get it by a shuffle.
// The waves are joined at the end.
template <int DP, bool BF16, bool FP8>
__device__ __forceinline__ void attend_few(const KArgs& ka, const Task& w, lds_char* sk, lds_char* sv) {
    constexpr int EB = FP8 ? 1 : 2, B = DP * EB;   // bytes of a row
    constexpr int LPR = B / 16, RPL = 64 / LPR;    // lanes of a row, rows of a load
    constexpr int NL = 32 / RPL;
    const KvLayout& kv = ka.a.kv;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Rows<DP, BF16, FP8> x;
    x.init(ka, w.keys, w.kvh, w.tok0, w.nrows, w.row0, w.k1, w.lim0);
    lds_char* lk = sk + wave * 32 * B;
    lds_char* lv = sv + wave * 32 * B;
    const char* kb0 = (const char*)ka.a.k_cache + (int64_t)w.kvh * kv.head_stride * EB;
    const char* vb0 = (const char*)ka.a.v_cache + (int64_t)w.kvh * kv.head_stride * EB;
    const uint32_t bstep = (uint32_t)(kv.block_stride * EB), sstep = (uint32_t)(kv.slot_stride * EB);
    const int row_bytes = kv.head_dim * EB;
    int32_t pid;
    uint32_t pat;
    auto look = [&](int kb) {
        const int i = kb + x.col;
        pid = -1;
        pat = 0;
        if (i < w.k1) pid = w.keys.page(kv, i, pat);
    };
    // byte offset of this lane's key in the cache, -1 if there is none
    int64_t koff, voff;
    auto offset = [&]() {
        const bool ok = (uint32_t)pid < (uint32_t)kv.num_blocks;
        return ok ? (int64_t)((uint64_t)(uint32_t)pid * bstep + (uint64_t)pat * sstep) : (int64_t)-1;
    };
    auto fetch = [&](const char* base, int64_t off, lds_char* to) {
#if defined(__HIP_DEVICE_COMPILE__)
        const uint32_t lo = (uint32_t)off, hi = (uint32_t)((uint64_t)off >> 32);
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const int r = n * RPL + x.lane / LPR;
            const int c = (x.lane % LPR) ^ (FP8 ? turn8<B>(r) : turn<B>(r));
            const int64_t o = (int64_t)(((uint64_t)(uint32_t)__shfl((int)hi, r) << 32) | (uint32_t)__shfl((int)lo, r));
            const char* src = o >= 0 && c * 16 < row_bytes ? base + o + c * 16 : (const char*)g_zeros;
            __builtin_amdgcn_global_load_lds(src, (lds_ptr)(to + n * 1024), 16, 0, 0);
        }
#endif
    };
    constexpr int STEP = kWaves * 32;
    int kb = w.k0 + wave * 32;
    bool bad = false;
    if (kb < w.k1) {
        look(kb);
        koff = voff = offset();
        fetch(kb0, koff, lk);
        fetch(vb0, voff, lv);
        look(kb + STEP);
    }
    x.ready();
    for (; kb < w.k1; kb += STEP) {
        const bool more = kb + STEP < w.k1;
        // Loads end in order.  After K of this group came at least V of it (and at
        // most one page id); after V, if there is a next group, its K.
        wait_loads<NL>();
        v16f st;
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i] = 0.f;
#pragma unroll
        for (int g = 0; g < DP / 32; ++g) {  // 32 elements: two matrix steps
            Frag8 f0, f1;
            if constexpr (FP8) {
                const v4u u = *(const __attribute__((address_space(3))) v4u*)(lk + x.col * B + ((2 * g + x.half) ^ turn8<B>(x.col)) * 16);
                f0.u = widen8<BF16>(u[0], u[1]);
                f1.u = widen8<BF16>(u[2], u[3]);
            } else {
                lds_char* at = lk + x.col * B + ((4 * g + 2 * x.half) ^ turn<B>(x.col)) * 16;
                f0.u = *(const __attribute__((address_space(3))) v4u*)at;
                f1.u = *(const __attribute__((address_space(3))) v4u*)(at + 16);
            }
            st = mfma32<BF16>(f0, x.q[2 * g], st);
            st = mfma32<BF16>(f1, x.q[2 * g + 1], st);
        }
        if (more) {
            koff = offset();
            wait_lds();  // the tile of K has been read
            fetch(kb0, koff, lk);
            look(kb + 2 * STEP);
        }
        x.prepare(st, kb);
        Frag8 p[2];
        x.weights(st, p);
        if (more) wait_loads<NL>();
        else wait_loads<0>();
        if (min(kb + 32, w.k1) > x.wseen) {  // some row does not see some of these keys
#pragma unroll 1
            for (int n = 0; n < NL; ++n) {
                auto at = (__attribute__((address_space(3))) v4u*)(lv + n * 1024 + x.lane * 16);
                const v4u u = *at, f = finite_of<BF16, FP8>(u);
                bad |= differ(f, u);
                *at = f;
            }
        }
        x.values_dense(lv, p);
        if (more) {
            wait_lds();  // the tile of V has been read
            fetch(vb0, koff, lv);
        }
    }
    x.l += __shfl_xor(x.l, 32);
    if (__any(bad)) x.add_nonfinite(ka, w.keys, w.kvh, x.wseen < w.k0 ? w.k0 : w.k0 + (x.wseen - w.k0) / 32 * 32, w.k0, w.k1, kWaves, wave);

    // Joining: waves 2 and 3 into 0 and 1, then 1 into 0.  A lane meets its own
    // counterpart, so the layout is the registers'.
    auto lo = (__attribute__((address_space(3))) float*)sk;
    typedef __attribute__((address_space(3))) v4f lds_v4f;
    constexpr int PER = (DP / 32 * 16 + 2) * 64;  // floats of a wave
#pragma unroll
    for (int n = 2; n >= 1; n >>= 1) {
        __syncthreads();
        if (wave >= n && wave < 2 * n) {
            auto o = lo + (wave - n) * PER;
            o[x.lane] = x.m;
            o[64 + x.lane] = x.l;
#pragma unroll
            for (int t = 0; t < DP / 32; ++t)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *(lds_v4f*)(o + 128 + ((t * 4 + g) * 64 + x.lane) * 4) =
                        v4f{x.acc[t][4 * g], x.acc[t][4 * g + 1], x.acc[t][4 * g + 2], x.acc[t][4 * g + 3]};
        }
        __syncthreads();
        if (wave < n) {
            auto o = lo + wave * PER;
            const float m2 = o[x.lane], to = fmaxf(x.m, m2);
            const float f1 = __builtin_amdgcn_exp2f(x.m - to), f2 = __builtin_amdgcn_exp2f(m2 - to);
            x.m = to;
            x.l = x.l * f1 + o[64 + x.lane] * f2;
#pragma unroll
            for (int t = 0; t < DP / 32; ++t)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const v4f y = *(const lds_v4f*)(o + 128 + ((t * 4 + g) * 64 + x.lane) * 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x.acc[t][4 * g + j] = x.acc[t][4 * g + j] * f1 + y[j] * f2;
                }
        }
    }
    if (wave == 0) x.store(ka, w.kvh, w.part, w.direct);
}

// ---------------------------------------------------------------------------
// many rows: tiles of keys shared by the waves
// ---------------------------------------------------------------------------

// Each wave has 32 rows of its own; tiles of 64 keys are staged in LDS for all
// four, in two buffers.  What bounds this is the matrix units and, with as many
// cycles, the exponentials, so a wave starts the score product of the next 32
// keys before it turns the last ones into weights.  K and V of the next tile
// travel one after the other, through the same registers.
template <int DP, bool BF16, bool FP8>
__device__ __forceinline__ void attend_many(const KArgs& ka, const Task& w, lds_char* sk, lds_char* sv) {
    constexpr int KT = 64;
    constexpr int EPC = FP8 ? 16 : 8, EB = FP8 ? 1 : 2;
    constexpr int NL = DP / 4 / EPC;        // 16-byte loads of a thread: a quarter of a row
    constexpr int KP = Padded<DP>::K, VP = Padded<DP>::V;
    typedef __attribute__((address_space(3))) v4u lds_v4u;
    const KvLayout& kv = ka.a.kv;
    const int tid = threadIdx.x, wave = tid >> 6;
    const int D = kv.head_dim;
    const int wrow0 = w.row0 + wave * kCols;
    const bool wlive = __builtin_amdgcn_readfirstlane(wrow0 < w.nrows);
    Rows<DP, BF16, FP8> x;
    x.init(ka, w.keys, w.kvh, w.tok0, w.nrows, wrow0, w.k1, w.lim0);
    // keys that every row of the workgroup sees
    const int gseen = min(w.k1, w.lim0 == kAll ? w.k1 : max(w.keys.shared, w.lim0 + (int)ka.per_group.div(w.row0)));

    // staging: four threads a row, chunk 4 n + tid % 4 of it
    const int sr = tid >> 2, sc = tid & 3;
    const char* kb0 = (const char*)ka.a.k_cache + (int64_t)w.kvh * kv.head_stride * EB;
    const char* vb0 = (const char*)ka.a.v_cache + (int64_t)w.kvh * kv.head_stride * EB;
    const uint32_t bstep = (uint32_t)(kv.block_stride * EB), sstep = (uint32_t)(kv.slot_stride * EB);
    v4u rg[NL];
    int32_t pid = -1;
    uint32_t pat = 0;
    uint64_t off = 0;
    bool ok = false;
    auto look = [&](int kt) {
        const int i = kt + sr;
        pid = -1;
        if (i < w.k1) pid = w.keys.page(kv, i, pat);
    };
    auto settle = [&]() {  // the offset of the row that was looked up
        ok = (uint32_t)pid < (uint32_t)kv.num_blocks;
        off = (uint64_t)(ok ? (uint32_t)pid : 0u) * bstep + (uint64_t)(ok ? pat : 0u) * sstep;
    };
    // What is no key of this workgroup, or beyond the head, reads the cache's first
    // elements instead and is zeroed before use: no load hides behind a branch.
    auto load = [&](const char* base) {
#pragma unroll
        for (int n = 0; n < NL; ++n) rg[n] = ld16(base + off + ((4 * n + sc) * EPC < D ? (4 * n + sc) * 16 : 0));
    };
    auto stage = [&](lds_char* to) {  // to: this thread's place in its row
        if (D < DP || !__all(ok)) {
#pragma unroll
            for (int n = 0; n < NL; ++n) rg[n] &= ok && (4 * n + sc) * EPC < D ? ~0u : 0u;
        }
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            if constexpr (FP8) {
                *(lds_v4u*)(to + 128 * n) = widen8<BF16>(rg[n][0], rg[n][1]);
                *(lds_v4u*)(to + 128 * n + 16) = widen8<BF16>(rg[n][2], rg[n][3]);
            } else {
                *(lds_v4u*)(to + 64 * n) = rg[n];
            }
        }
    };
    bool bad = false;
    auto stage_v = [&](int kt, lds_char* to) {
        if (min(kt + KT, w.k1) > gseen) {  // some row does not see some of these keys
#pragma unroll
            for (int n = 0; n < NL; ++n) {
                const v4u f = finite_of<BF16, FP8>(rg[n]);
                bad |= ok && differ(f, rg[n]);
                rg[n] = f;
            }
        }
        stage(to);
    };
    auto scores = [&](lds_char* k, v16f& st) {  // k: this lane's row and half
#pragma unroll
        for (int i = 0; i < 16; ++i) st[i] = 0.f;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            Frag8 kf;
            kf.u = *(const lds_v4u*)(k + 64 * (s >> 1) + 16 * (s & 1));
            st = mfma32<BF16>(kf, x.q[s], st);
        }
    };
    lds_char* const put_k = sk + sr * KP + sc * (FP8 ? 32 : 16);
    lds_char* const put_v = sv + sr * VP + sc * (FP8 ? 32 : 16);
    lds_char* const get_k = sk + x.col * KP + 32 * x.half;
    v16f s0, s1;
    Frag8 p[2];
    if (w.k0 < w.k1) look(w.k0);
    x.ready();
    if (w.k0 < w.k1) {
        settle();
        load(kb0);
        stage(put_k);
        load(vb0);
        look(w.k0 + KT);
        stage_v(w.k0, put_v);
        settle();
        load(kb0);
        __syncthreads();
        if (wlive) {
            scores(get_k, s0);
            x.prepare(s0, w.k0);
        }
    }
    // Tile kt from one buffer while tile kt + 64 comes into the other.  On entry:
    // the scores of its first 32 keys, and K of the next tile in registers.
    auto step = [&](int kt, int kc, int vc, int kn, int vn) {
        const bool more = kt + KT < w.k1;
        if (more) {
            stage(put_k + kn);
            load(vb0);
            look(kt + 2 * KT);
        }
        if (wlive) {
            scores(get_k + kc + 32 * KP, s1);
            x.weights(s0, p);
            x.values_padded(sv + vc, p);
            x.prepare(s1, kt + 32);
        }
        __syncthreads();  // K of the next tile is there
        if (more) {
            stage_v(kt + KT, put_v + vn);
            settle();
            load(kb0);
        }
        if (wlive) {
            if (more) scores(get_k + kn, s0);
            x.weights(s1, p);
            x.values_padded(sv + vc + 32 * VP, p);
            if (more) x.prepare(s0, kt + KT);
        }
        __syncthreads();  // V of the next tile is there, and this tile is done with
    };
    for (int kt = w.k0; kt < w.k1; kt += 2 * KT) {
        step(kt, 0, 0, KT * KP, KT * VP);
        if (kt + KT < w.k1) step(kt + KT, KT * KP, KT * VP, 0, 0);
    }
    x.l += __shfl_xor(x.l, 32);
    if (__syncthreads_or(bad) && wlive) x.add_nonfinite(ka, w.keys, w.kvh, gseen < w.k0 ? w.k0 : w.k0 + (gseen - w.k0) / KT * KT, w.k0, w.k1, 1, 0);
    x.store(ka, w.kvh, w.part, w.direct);
}

// A unit of a segment whose workgroups come in groups of `tiles` that read the
// same keys: whole groups go to one XCD (workgroup ids alternate between the 8
// XCDs), so that the group's keys are fetched into one L2 only.
__device__ __forceinline__ bool grouped_unit(int64_t id, int64_t groups, int tiles, int64_t& group, int& tile) {
    if (groups % 8 == 0 || groups >= 32) {
        const int64_t j = id >> 3;
        group = (j / tiles) * 8 + (id & 7);
        tile = (int)(j % tiles);
        return group < groups;
    }
    group = id / tiles;
    tile = (int)(id % tiles);
    return true;
}

template <int DP, bool BF16, bool FP8>
__global__ __launch_bounds__(kThreads, DP == 256 ? 1 : 2) void attn_kernel(KArgs ka) {
    // two tiles of 64 padded rows of K and of V, or four waves' 32 dense rows (and then two waves' results in s_k)
    __shared__ __attribute__((aligned(16))) char s_k[2 * 64 * Padded<DP>::K], s_v[2 * 64 * Padded<DP>::V];
    const AttnArgs& a = ka.a;
    const Plan& p = ka.p;
    int64_t id = blockIdx.x;
    const bool direct = p.parts == 1;
    const int heads = a.kv.kv_heads;
    bool few;
    int kvh, part, base, row0, rows, k1, lim0;
    int64_t tok0, k0;
    Keys keys{a.prefix_table, nullptr, (int)a.prefix_len};
    if (id < p.pre_units) {
        int64_t group;
        int tile;
        if (!grouped_unit(id, (int64_t)heads * p.pre_parts, p.pre_tiles, group, tile)) return;
        few = p.pre_few;
        kvh = (int)(group % heads);
        part = (int)(group / heads);
        base = 0;
        row0 = tile * kRowsWide;
        rows = (int)a.T * ka.G;
        tok0 = 0;
        k0 = (int64_t)part * p.pre_chunk;
        k1 = (int)min(k0 + p.pre_chunk, a.prefix_len);
        lim0 = kAll;
    } else {
        id -= p.pre_units;
        few = id < p.few_units;
        int r, tile = 0;
        if (few) {
            part = (int)(id % p.few_parts);
            const int64_t g = id / p.few_parts;
            kvh = (int)(g % heads);
            r = (int)(g / heads);
        } else {
            int64_t group;
            if (!grouped_unit(id - p.few_units, a.B * heads * p.many_parts, p.many_tiles, group, tile)) return;
            tile = p.many_tiles - 1 - tile;  // the last rows see the most keys: first
            part = (int)(group % p.many_parts);
            group /= p.many_parts;
            kvh = (int)(group % heads);
            r = (int)(group / heads);
        }
        int64_t t0 = a.cu[r], t1 = a.cu[r + 1];
        t0 = t0 < 0 ? 0 : t0;
        t1 = t1 > a.T ? a.T : t1;
        const int n = t1 > t0 ? (int)min(t1 - t0, a.max_new) : 0;
        tok0 = t0;
        rows = n * ka.G;
        row0 = tile * kRowsWide;
        if (few != (rows <= kCols) || row0 >= rows) return;
        int64_t len = a.kv_lens[r];
        len = len < 0 ? 0 : min(min(len, a.max_kv), a.max_blocks * a.kv.block_size);
        keys.own = a.block_table + (int64_t)r * a.max_blocks;
        keys.shared = p.joint ? (int)a.prefix_len : 0;
        lim0 = keys.shared + (int)len - n + 1;
        const int chunk = few ? p.few_chunk : p.many_chunk;
        const int last = min(row0 + (few ? kCols : kRowsWide), rows) - 1;
        const int end = max(keys.shared, lim0 + (int)ka.per_group.div(last));  // keys that the tile's last row sees
        k0 = (int64_t)part * chunk;
        base = p.pre_parts;
        // how many parts each token's own keys have, for the join
        if (!direct && part == 0 && kvh == 0)
            for (int i = threadIdx.x; i <= last - row0; i += kThreads) {
                const int t = (int)ka.per_group.div(row0 + i);
                ka.part_n[t0 + t] = (max(keys.shared, lim0 + t) + chunk - 1) / chunk;
            }
        if (k0 >= end && !(direct && part == 0)) return;
        k1 = (int)min(k0 + chunk, (int64_t)end);
    }
    const Task w{keys, kvh, rows, row0, (int)k0, k1, lim0, base + part, tok0, direct};
    if (few) attend_few<DP, BF16, FP8>(ka, w, (lds_char*)s_k, (lds_char*)s_v);
    else attend_many<DP, BF16, FP8>(ka, w, (lds_char*)s_k, (lds_char*)s_v);
}

// Joins the parts of every row: D / 4 threads a row.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(KArgs ka) {
    const AttnArgs& a = ka.a;
    const int D = a.kv.head_dim, tpr = D / 4, rpw = kThreads / tpr;
    const int sub = threadIdx.x / tpr, d4 = threadIdx.x % tpr;
    const int64_t row = (int64_t)blockIdx.x * rpw + sub, rows = a.T * a.q_heads;
    if (sub >= rpw || row >= rows) return;
    const int64_t tok = row / a.q_heads;
    if (tok >= a.cu[a.B]) return;
    int own = ka.part_n[tok];
    own = own < 0 ? 0 : own > ka.p.own_parts ? ka.p.own_parts : own;
    const int n = ka.p.pre_parts + own;
    float mm = kNone;
    for (int p = 0; p < n; ++p) mm = fmaxf(mm, ka.part_m[(int64_t)p * rows + row]);
    float ll = 0.f;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < n; ++p) {
        const int64_t at = (int64_t)p * rows + row;
        const float f = __builtin_amdgcn_exp2f(ka.part_m[at] - mm);
        ll += f * ka.part_l[at];
        const v4f x = *(const v4f*)(ka.part_o + at * D + 4 * d4);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += f * x[j];
    }
    const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
    const int64_t hd = row - tok * a.q_heads;
    const uint32_t w0 = pack2<BF16>(o[0] * inv, o[1] * inv);
    const uint32_t w1 = pack2<BF16>(o[2] * inv, o[3] * inv);
    *(uint2*)((uint16_t*)a.out + tok * a.out_stride + hd * D + 4 * d4) = make_uint2(w0, w1);
    if (a.lse && d4 == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

static int pad_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

static Plan make_plan(const AttnArgs& a) {
    Plan p{};
    const int64_t hk = a.kv.kv_heads, G = a.q_heads / hk;
    const int64_t rows = a.T * G;
    const int64_t slots = pad_dim(a.kv.head_dim) == 256 ? 256 : 512;  // workgroups that run at once
    const int64_t own = a.total_kv > 0 ? a.total_kv : a.B * a.max_kv;
    const int64_t P = a.prefix_len;
    const bool many = a.max_new * G > kCols;
    // a request whose rows fill tiles by themselves gains nothing from sharing,
    // nor does a prefix that is short beside the own keys
    p.joint = P > 0 && (a.B == 1 || rows >= a.B * kRowsWide || P * (a.B - 1) <= own / 4);
    const int64_t extra = p.joint ? P : 0;
    const int64_t pre_keys = p.joint ? 0 : P;
    if (pre_keys) {
        p.pre_few = rows <= kCols;
        p.pre_tiles = p.pre_few ? 1 : (int)cdiv(rows, kRowsWide);
    }
    // keys of a workgroup so that the card is filled about once
    const int64_t own_tiles = many ? cdiv(rows, kRowsWide) + a.B : a.B;
    const int64_t own_keys = own + extra * a.B;
    const int64_t all = hk * (pre_keys * p.pre_tiles + (many ? own_keys / (a.B ? a.B : 1) * own_tiles : own_keys));
    int64_t per = cdiv(cdiv(all, slots), 128) * 128;
    if (per < 256) per = 256;
    if (pre_keys) {
        p.pre_parts = (int)cdiv(pre_keys, per);
        p.pre_chunk = (int)(cdiv(cdiv(pre_keys, p.pre_parts), 64) * 64);
        p.pre_parts = (int)cdiv(pre_keys, p.pre_chunk);
        const int64_t groups = hk * p.pre_parts;
        p.pre_units = (groups % 8 == 0 || groups >= 32 ? cdiv(groups, 8) * 8 : groups) * p.pre_tiles;
    }
    const int64_t longest = a.max_kv + extra;
    int64_t parts = cdiv(longest, per);
    if (parts < 1) parts = 1;
    p.few_parts = (int)parts;
    p.few_chunk = (int)(cdiv(cdiv(longest > 0 ? longest : 1, parts), 128) * 128);
    p.few_parts = (int)(longest > 0 ? cdiv(longest, p.few_chunk) : 1);
    p.few_units = a.B * hk * p.few_parts;
    if (many) {
        p.many_chunk = p.few_chunk;
        p.many_parts = p.few_parts;
        p.many_tiles = (int)cdiv(a.max_new * G, kRowsWide);
        const int64_t groups = a.B * hk * p.many_parts;
        p.many_units = (groups % 8 == 0 || groups >= 32 ? cdiv(groups, 8) * 8 : groups) * p.many_tiles;
    }
    p.own_parts = p.few_parts > p.many_parts ? p.few_parts : p.many_parts;
    p.parts = p.pre_parts + p.own_parts;
    return p;
}

static size_t up256(size_t b) { return (b + 255) / 256 * 256; }

static int64_t units_of(const Plan& p) { return p.pre_units + p.few_units + p.many_units; }

size_t attn_workspace(const AttnArgs& a) {
    const Plan p = make_plan(a);
    if (units_of(p) >= (int64_t)1 << 24) return SIZE_MAX;
    if (p.parts == 1) return 0;
    const size_t rows = (size_t)a.T * a.q_heads;
    return up256((size_t)p.parts * rows * a.kv.head_dim * 4) + 2 * up256((size_t)p.parts * rows * 4) + up256((size_t)a.T * 4);
}

template <int DP, bool BF16, bool FP8>
static hipError_t launch_one(const KArgs& ka, int64_t units) {
    if (plan_recorder()) {
        plan_record("attn<%d,%s,%s> grid=%lld prefix=%d few=%d many=%d joint=%d", DP, BF16 ? "bf16" : "fp16", FP8 ? "e4m3" : "16",
                    (long long)units, ka.p.pre_parts, ka.p.few_parts, ka.p.many_parts, (int)ka.p.joint);
        return hipSuccess;
    }
    hipLaunchKernelGGL((attn_kernel<DP, BF16, FP8>), dim3((unsigned)units), dim3(kThreads), 0, ka.a.stream, ka);
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
    ka.p = make_plan(a);
    ka.G = a.q_heads / a.kv.kv_heads;
    ka.per_group = FastDiv::of((uint32_t)ka.G);
    if (ka.p.parts > 1) {
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
    const int64_t units = units_of(ka.p);
    if (units < 1 || units >= (int64_t)1 << 24) return hipErrorInvalidConfiguration;
    const int dp = pad_dim(a.kv.head_dim);
    hipError_t e = dp == 64 ? launch_dim<64>(ka, units) : dp == 128 ? launch_dim<128>(ka, units) : launch_dim<256>(ka, units);
    if (e != hipSuccess || ka.p.parts == 1) return e;
    const int rpw = kThreads / (a.kv.head_dim / 4);
    const int64_t wgs = cdiv(a.T * a.q_heads, rpw);
    if (plan_recorder()) {
        plan_record("attn_join<%s> grid=%lld parts=%d", a.bf16 ? "bf16" : "fp16", (long long)wgs, ka.p.parts);
        return hipSuccess;
    }
    if (a.bf16) hipLaunchKernelGGL((attn_join_kernel<true>), dim3((unsigned)wgs), dim3(kThreads), 0, a.stream, ka);
    else hipLaunchKernelGGL((attn_join_kernel<false>), dim3((unsigned)wgs), dim3(kThreads), 0, a.stream, ka);
    return hipGetLastError();
}

}  // namespace hq
