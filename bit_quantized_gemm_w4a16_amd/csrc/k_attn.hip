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

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 32;                       // query rows of a wave's matrix tile
constexpr int kRowsWide = kWaves * kCols;       // rows of a workgroup whose waves take different rows
constexpr float kNone = -3.0e38f;               // running maximum before any key
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

// Byte offset of 16-byte chunk c of key row r in a tile of rows of DP 16-bit
// elements.  K: lanes of a load read one chunk of 32 rows, so the rows' chunks
// are spread over all banks.  V: a transposing load reads 4 rows times 4
// neighbouring chunks, which are spread instead.
template <int DP>
__device__ __forceinline__ int k_at(int r, int c) {
    const int x = DP == 64 ? (r >> 1) & 7 : r & 15;
    return r * DP * 2 + ((c ^ x) << 4);
}
template <int DP>
__device__ __forceinline__ int v_at(int r, int c) {
    const int x = DP == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
    return r * DP * 2 + ((c ^ x) << 4);
}

template <bool BF16>
__device__ __forceinline__ void widen8(uint32_t lo, uint32_t hi, v4u& o) {  // 8 E4M3 codes -> 16-bit values (exact)
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
}

// Zeroes the elements of u whose exponent is all ones; true if there were any.
template <bool BF16>
__device__ __forceinline__ bool drop_nonfinite(v4u& u) {
    constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((u[i] & E) == E) {
            u[i] &= 0xFFFF0000u;
            any = true;
        }
        if ((u[i] & (E << 16)) == (E << 16)) {
            u[i] &= 0x0000FFFFu;
            any = true;
        }
    }
    return any;
}

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

// ---------------------------------------------------------------------------
// one workgroup's rows times keys
// ---------------------------------------------------------------------------

// FEW: the waves share the rows and split each tile of 128 keys; else they
// share a tile of 64 keys and split the rows.
template <int DP, bool BF16, bool FP8, bool FEW>
__device__ __forceinline__ void attend(const KArgs& ka, const Keys keys, int kvh, int64_t tok0, int nrows, int row0, int k0, int k1,
                       int lim0, int part, int part_base, bool direct, char* lds) {
    constexpr int KT = FEW ? 128 : 64;
    constexpr int SUB = FEW ? 1 : 2;               // 32-key groups of a tile that a wave takes
    constexpr int EPC = FP8 ? 16 : 8;              // elements of a 16-byte load
    constexpr int CPR = DP / EPC;                  // loads per key row
    constexpr int RPP = kThreads / CPR;            // key rows of one pass
    constexpr int NP = KT / RPP;
    constexpr int KS = DP / 16, DT = DP / 32;
    const AttnArgs& a = ka.a;
    const KvLayout& kv = a.kv;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int half = lane >> 5, col = lane & 31;
    const int D = kv.head_dim;
    char* lk = lds;
    char* lv = lds + KT * DP * 2;

    // this lane's query row
    const int row = row0 + (FEW ? 0 : wave * kCols) + col;
    const bool live = row < nrows;
    const int rtok = live ? (int)ka.per_group.div(row) : 0;
    const int64_t tok = tok0 + rtok;
    const int head = kvh * ka.G + (live ? row - rtok * ka.G : 0);
    // lim0: keys that the first token of the request sees (INT_MAX: every row sees all)
    const int lim = lim0 == 0x7FFFFFFF ? k1 : max(keys.shared, lim0 + rtok);
    const int wrow0 = row0 + (FEW ? 0 : wave * kCols);
    const bool wlive = wrow0 < nrows;
    // keys that every live row of this wave / workgroup sees
    const int wtok = (int)ka.per_group.div(wlive ? wrow0 : 0);
    const int wlim = lim0 == 0x7FFFFFFF ? k1 : max(keys.shared, lim0 + wtok);
    const int glim = lim0 == 0x7FFFFFFF ? k1 : max(keys.shared, lim0 + (int)ka.per_group.div(row0));

    Frag8 qf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int d = 16 * s + 8 * half;
        qf[s].u = v4u{0u, 0u, 0u, 0u};
        if (live && d < D) qf[s].u = ld16((const uint16_t*)a.q + tok * a.q_stride + (int64_t)head * D + d);
    }
    const float ksc = FP8 ? a.k_scale[kvh] : 1.f;
    const float vsc = FP8 ? a.v_scale[kvh] : 1.f;
    // s = x.k * c1, or with a cap s = c2 tanh(x.k * c1)
    const bool cap = a.softcap > 0.f;
    const float c1 = cap ? a.scale * ksc / a.softcap : a.scale * ksc * kLog2e;
    const float c2 = a.softcap * kLog2e;

    v16f acc[DT];
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
    float m = kNone, l = 0.f;

    // staging: this thread loads 16-byte chunk cc of rows cr, cr + RPP, ...
    const int cr = tid / CPR, cc = tid % CPR;
    const bool cin = cc * EPC < D;
    const char* kbase = (const char*)a.k_cache + ((int64_t)kvh * kv.head_stride + cc * EPC) * (FP8 ? 1 : 2);
    const char* vbase = (const char*)a.v_cache + ((int64_t)kvh * kv.head_stride + cc * EPC) * (FP8 ? 1 : 2);
    v4u rk[NP], rv[NP];
    auto load = [&](int kt) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int i = kt + p * RPP + cr;
            rk[p] = rv[p] = v4u{0u, 0u, 0u, 0u};
            if (i < k1 && cin) {
                uint32_t at;
                const int32_t b = keys.page(kv, i, at);
                if (b >= 0 && b < kv.num_blocks) {
                    const int64_t off = ((int64_t)b * kv.block_stride + (int64_t)at * kv.slot_stride) * (FP8 ? 1 : 2);
                    rk[p] = ld16(kbase + off);
                    rv[p] = ld16(vbase + off);
                }
            }
        }
    };
    __shared__ int s_bad;  // a value that some row does not see is not finite
    if (tid == 0) s_bad = 0;

    if (k0 < k1) load(k0);
    for (int kt = k0; kt < k1; kt += KT) {
        const bool masked = min(kt + KT, k1) > glim;  // some row does not see some key of this tile
        __syncthreads();                     // the last tile's reads are done
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int r = p * RPP + cr;
            if constexpr (FP8) {
                v4u x, y;
                widen8<BF16>(rk[p][0], rk[p][1], x);
                widen8<BF16>(rk[p][2], rk[p][3], y);
                *(v4u*)(lk + k_at<DP>(r, 2 * cc)) = x;
                *(v4u*)(lk + k_at<DP>(r, 2 * cc + 1)) = y;
                widen8<BF16>(rv[p][0], rv[p][1], x);
                widen8<BF16>(rv[p][2], rv[p][3], y);
                if (masked) {
                    const bool bx = drop_nonfinite<BF16>(x), by = drop_nonfinite<BF16>(y);
                    if (bx || by) s_bad = 1;
                }
                *(v4u*)(lv + v_at<DP>(r, 2 * cc)) = x;
                *(v4u*)(lv + v_at<DP>(r, 2 * cc + 1)) = y;
            } else {
                *(v4u*)(lk + k_at<DP>(r, cc)) = rk[p];
                v4u x = rv[p];
                if (masked && drop_nonfinite<BF16>(x)) s_bad = 1;
                *(v4u*)(lv + v_at<DP>(r, cc)) = x;
            }
        }
        __syncthreads();
        if (kt + KT < k1) load(kt + KT);
        if (!wlive) continue;

        // S^T: rows are keys, columns are queries
        v16f st[SUB];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            const int kr = (FEW ? wave * 32 : u * 32) + col;
#pragma unroll
            for (int i = 0; i < 16; ++i) st[u][i] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                Frag8 kf;
                kf.u = *(const v4u*)(lk + k_at<DP>(kr, 2 * s + half));
                if constexpr (BF16) st[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf.b, qf[s].b, st[u], 0, 0, 0);
                else st[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf.h, qf[s].h, st[u], 0, 0, 0);
            }
        }
        // register i of group u is key kb + 32 u + 8 (i / 4) + 4 half + i % 4
        const int kb = kt + (FEW ? wave * 32 : 0);
        float mx = m;
        const bool edge = kb + 32 * SUB > min(wlim, k1);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = st[u][i] * c1;
                if (cap) s = c2 * (1.f - 2.f / (1.f + __builtin_amdgcn_exp2f(2.f * kLog2e * s)));
                if (edge) {
                    const int key = kb + 32 * u + 8 * (i >> 2) + 4 * half + (i & 3);
                    if (key >= min(lim, k1)) s = -INFINITY;
                }
                st[u][i] = s;
                mx = fmaxf(mx, s);
            }
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float shrink = __builtin_amdgcn_exp2f(m - mx);
        m = mx;
        l *= shrink;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[t][i] *= shrink;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                st[u][i] = __builtin_amdgcn_exp2f(st[u][i] - m);
                l += st[u][i];
            }
        // O^T += V^T P^T, 16 keys at a time
        const int i16 = lane & 15, dsel = (lane >> 4) & 1;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                Frag8 pf;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    pf.u[j] = (uint32_t)f32_to_16<BF16>(st[u][8 * ks + 2 * j]) |
                              ((uint32_t)f32_to_16<BF16>(st[u][8 * ks + 2 * j + 1]) << 16);
                const int vr = (FEW ? wave * 32 : u * 32) + 16 * ks + 4 * half + (i16 >> 2);
#pragma unroll
                for (int t = 0; t < DT; ++t) {
#if defined(__HIP_DEVICE_COMPILE__)
                    const int ch = 4 * t + 2 * dsel + ((i16 & 3) >> 1), in = (i16 & 1) * 8;
                    Frag8 vf;
                    const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(lv + v_at<DP>(vr, ch) + in));
                    const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(lv + v_at<DP>(vr + 8, ch) + in));
                    const v2u xu = __builtin_bit_cast(v2u, x), yu = __builtin_bit_cast(v2u, y);
                    vf.u = v4u{xu[0], xu[1], yu[0], yu[1]};
                    if constexpr (BF16) acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf.b, pf.b, acc[t], 0, 0, 0);
                    else acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf.h, pf.h, acc[t], 0, 0, 0);
#endif
                }
            }
    }
    l += __shfl_xor(l, 32);
    __syncthreads();  // the last tile's reads are done, s_bad is final

    // Values that are not finite were left out of the tiles where some row does
    // not see them (0 times infinity would reach that row).  The rows that do
    // see one get it here: with its weight, which is positive, it can only make
    // the sum that infinity or NaN.
    if (s_bad && wlive && (!FEW || wave == 0)) {
        const int first = glim < k0 ? k0 : k0 + (glim - k0) / KT * KT;
        for (int key = first; key < k1; ++key) {
            uint32_t at;
            const int32_t b = keys.page(kv, key, at);
            if (b < 0 || b >= kv.num_blocks || key >= lim) continue;
            const int64_t off = (int64_t)b * kv.block_stride + (int64_t)at * kv.slot_stride + (int64_t)kvh * kv.head_stride;
#pragma unroll
            for (int t = 0; t < DT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int d = 32 * t + 8 * (i >> 2) + 4 * half + (i & 3);
                    if (d >= D) continue;
                    float v;
                    if constexpr (FP8) v = (((const uint8_t*)a.v_cache)[off + d] & 0x7Fu) == 0x7Fu ? __builtin_nanf("") : 0.f;
                    else v = bits16_to_f32<BF16>(((const uint16_t*)a.v_cache)[off + d]);
                    if (!(fabsf(v) < INFINITY)) acc[t][i] += v;
                }
        }
    }

    if constexpr (FEW) {
        // join the four waves' keys
        float* lo = (float*)lds;                               // [wave][32 rows][DP]
        __shared__ float s_m[kWaves][kCols], s_l[kWaves][kCols];
        if (half == 0) {
            s_m[wave][col] = m;
            s_l[wave][col] = l;
        }
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *(v4f*)(lo + (wave * kCols + col) * DP + (((32 * t + 8 * g + 4 * half) / 4) ^ (col & 7)) * 4) =
                    v4f{acc[t][4 * g], acc[t][4 * g + 1], acc[t][4 * g + 2], acc[t][4 * g + 3]};
        __syncthreads();
        for (int i = tid; i < kCols * DP / 4; i += kThreads) {
            const int r = i / (DP / 4), d4 = i % (DP / 4);
            if (row0 + r >= nrows || d4 * 4 >= D) continue;
            float mm = kNone, ll = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][r]);
            v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(s_m[w][r] - mm);
                ll += f * s_l[w][r];
                const v4f x = *(const v4f*)(lo + (w * kCols + r) * DP + (d4 ^ (r & 7)) * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += f * x[j];
            }
            const int rt = (int)ka.per_group.div(row0 + r), hd = kvh * ka.G + (row0 + r - rt * ka.G);
            const int64_t tk = tok0 + rt;
            if (direct) {
                const float inv = ll > 0.f || ll != ll ? vsc / ll : 0.f;
                uint32_t w0 = (uint32_t)f32_to_16<BF16>(o[0] * inv) | ((uint32_t)f32_to_16<BF16>(o[1] * inv) << 16);
                uint32_t w1 = (uint32_t)f32_to_16<BF16>(o[2] * inv) | ((uint32_t)f32_to_16<BF16>(o[3] * inv) << 16);
                *(uint2*)((uint16_t*)a.out + tk * a.out_stride + (int64_t)hd * D + 4 * d4) = make_uint2(w0, w1);
                if (a.lse && d4 == 0) a.lse[tk * a.q_heads + hd] = ll == 0.f ? -INFINITY : (mm + __builtin_amdgcn_logf(ll)) * kLn2;
            } else {
                const int64_t pr = ((int64_t)(part_base + part) * a.T + tk) * a.q_heads + hd;
                *(v4f*)(ka.part_o + pr * D + 4 * d4) = o * vsc;
                if (d4 == 0) {
                    ka.part_m[pr] = mm;
                    ka.part_l[pr] = ll;
                }
            }
        }
    } else if (live) {
        const int64_t pr = ((int64_t)(part_base + part) * a.T + tok) * a.q_heads + head;
        const float inv = !direct ? vsc : l > 0.f || l != l ? vsc / l : 0.f;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int d = 32 * t + 8 * g + 4 * half;
                if (d >= D) continue;
                v4f o;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = acc[t][4 * g + j] * inv;
                if (direct) {
                    uint32_t w0 = (uint32_t)f32_to_16<BF16>(o[0]) | ((uint32_t)f32_to_16<BF16>(o[1]) << 16);
                    uint32_t w1 = (uint32_t)f32_to_16<BF16>(o[2]) | ((uint32_t)f32_to_16<BF16>(o[3]) << 16);
                    *(uint2*)((uint16_t*)a.out + tok * a.out_stride + (int64_t)head * D + d) = make_uint2(w0, w1);
                } else {
                    *(v4f*)(ka.part_o + pr * D + d) = o;
                }
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
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const AttnArgs& a = ka.a;
    const Plan& p = ka.p;
    int64_t id = blockIdx.x;
    const bool direct = p.parts == 1;
    Keys keys{a.prefix_table, nullptr, 0};
    if (id < p.pre_units) {
        int64_t group;
        int tile;
        if (!grouped_unit(id, (int64_t)a.kv.kv_heads * p.pre_parts, p.pre_tiles, group, tile)) return;
        const int kvh = (int)(group % a.kv.kv_heads), part = (int)(group / a.kv.kv_heads);
        const int k0 = part * p.pre_chunk, k1 = min(k0 + p.pre_chunk, (int)a.prefix_len);
        keys.shared = (int)a.prefix_len;
        const int rows = (int)a.T * ka.G;
        if (p.pre_few) attend<DP, BF16, FP8, true>(ka, keys, kvh, 0, rows, 0, k0, k1, 0x7FFFFFFF, part, 0, direct, lds);
        else attend<DP, BF16, FP8, false>(ka, keys, kvh, 0, rows, tile * kRowsWide, k0, k1, 0x7FFFFFFF, part, 0, direct, lds);
        return;
    }
    id -= p.pre_units;
    const bool few = id < p.few_units;
    int r, kvh, part, tile = 0;
    if (few) {
        part = (int)(id % p.few_parts);
        const int64_t g = id / p.few_parts;
        kvh = (int)(g % a.kv.kv_heads);
        r = (int)(g / a.kv.kv_heads);
    } else {
        id -= p.few_units;
        int64_t group;
        if (!grouped_unit(id, a.B * a.kv.kv_heads * p.many_parts, p.many_tiles, group, tile)) return;
        tile = p.many_tiles - 1 - tile;  // the last rows see the most keys: first
        part = (int)(group % p.many_parts);
        group /= p.many_parts;
        kvh = (int)(group % a.kv.kv_heads);
        r = (int)(group / a.kv.kv_heads);
    }
    int64_t t0 = a.cu[r], t1 = a.cu[r + 1];
    t0 = t0 < 0 ? 0 : t0;
    t1 = t1 > a.T ? a.T : t1;
    const int n = t1 > t0 ? (int)min(t1 - t0, a.max_new) : 0;
    const int rows = n * ka.G;
    if (rows == 0 || few != (rows <= kCols)) return;
    const int row0 = few ? 0 : tile * kRowsWide;
    if (row0 >= rows) return;
    int64_t len = a.kv_lens[r];
    len = len < 0 ? 0 : min(min(len, a.max_kv), a.max_blocks * a.kv.block_size);
    keys.own = a.block_table + (int64_t)r * a.max_blocks;
    keys.shared = p.joint ? (int)a.prefix_len : 0;
    const int lim0 = keys.shared + (int)len - n + 1;
    const int chunk = few ? p.few_chunk : p.many_chunk;
    const int last = min(row0 + (few ? kCols : kRowsWide), rows) - 1;
    const int end = max(keys.shared, lim0 + (int)ka.per_group.div(last));  // keys that the tile's last row sees
    const int64_t k0 = (int64_t)part * chunk;
    // how many parts each token's own keys have, for the join
    if (!direct && part == 0 && kvh == 0)
        for (int i = threadIdx.x; i <= last - row0; i += kThreads) {
            const int t = (int)ka.per_group.div(row0 + i);
            const int e = max(keys.shared, lim0 + t);
            ka.part_n[t0 + t] = (e + chunk - 1) / chunk;
        }
    if (k0 >= end && !(direct && part == 0)) return;
    const int k1 = (int)min(k0 + chunk, (int64_t)end);
    const int base = p.pre_parts;
    if (few) attend<DP, BF16, FP8, true>(ka, keys, kvh, t0, rows, row0, (int)k0, k1, lim0, part, base, direct, lds);
    else attend<DP, BF16, FP8, false>(ka, keys, kvh, t0, rows, row0, (int)k0, k1, lim0, part, base, direct, lds);
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
    const uint32_t w0 = (uint32_t)f32_to_16<BF16>(o[0] * inv) | ((uint32_t)f32_to_16<BF16>(o[1] * inv) << 16);
    const uint32_t w1 = (uint32_t)f32_to_16<BF16>(o[2] * inv) | ((uint32_t)f32_to_16<BF16>(o[3] * inv) << 16);
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
static hipError_t launch_one(const KArgs& ka, int64_t units, size_t shared) {
    if (plan_recorder()) {
        plan_record("attn<%d,%s,%s> grid=%lld prefix=%d few=%d many=%d joint=%d", DP, BF16 ? "bf16" : "fp16", FP8 ? "e4m3" : "16",
                    (long long)units, ka.p.pre_parts, ka.p.few_parts, ka.p.many_parts, (int)ka.p.joint);
        return hipSuccess;
    }
    // allow dynamic LDS beyond the 64 KB default, once per instantiation
    static const hipError_t attr = hipFuncSetAttribute((const void*)attn_kernel<DP, BF16, FP8>,
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (attr != hipSuccess) return attr;
    hipLaunchKernelGGL((attn_kernel<DP, BF16, FP8>), dim3((unsigned)units), dim3(kThreads), shared, ka.a.stream, ka);
    return hipGetLastError();
}

template <int DP>
static hipError_t launch_dim(const KArgs& ka, int64_t units) {
    const size_t shared = (size_t)128 * DP * 4;
    const bool fp8 = ka.a.kv.dtype == HQ_DT_FP8_E4M3;
    if (ka.a.bf16) return fp8 ? launch_one<DP, true, true>(ka, units, shared) : launch_one<DP, true, false>(ka, units, shared);
    return fp8 ? launch_one<DP, false, true>(ka, units, shared) : launch_one<DP, false, false>(ka, units, shared);
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
