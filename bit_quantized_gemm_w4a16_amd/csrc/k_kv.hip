// Slot maps, rotary table, and the rotation of new tokens with their write to
// the paged key/value cache.
#include "hq_device.hpp"
#include "hq_internal.h"
#include "hq_kv.h"

namespace hq {

// ---------------------------------------------------------------------------
// block tables and slot maps
// ---------------------------------------------------------------------------

__device__ __forceinline__ int32_t sat_add(int32_t a, int32_t b) {  // a, b >= 0
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int32_t)s;
}

// Largest r with first[r] <= i, for first[0] = 0, nondecreasing, r < n: the
// owner of item i (requests without items share their offset with the next).
__device__ __forceinline__ int owner_of(const int32_t* first, int n, int32_t i) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Every workgroup makes the two prefix sums over the requests (new tokens, and
// the pages they need beyond the ones held) for itself in LDS: with at most
// 4096 requests that is a few KB from L2, less than a second launch would cost.
// It then writes its share of the tokens, the new table entries and the
// per-request outputs; each token and each new page finds its request by
// bisection.  A page taken in this very call is looked up in free_blocks, not in
// the table, so no workgroup waits for another.  Nothing but latency bounds it:
// lengths, sums, bisection, table entry, store (8 requests 2.8 us, 1500 requests
// with 42 thousand tokens 6.7 us).
constexpr int kSlotThreads = 512;

// Pages that the first n tokens of a request take.
__device__ __forceinline__ int32_t pages_of(const FastDiv& per_block, int32_t n) { return n ? (int32_t)per_block.div(n - 1) + 1 : 0; }

__global__ __launch_bounds__(kSlotThreads) void kv_slots_kernel(KvSlotsArgs a) {
    // cached tokens; new tokens, then their exclusive sums; the same of new pages
    __shared__ int32_t s_c[HQ_KV_MAX_REQUESTS], s_cu[HQ_KV_MAX_REQUESTS + 1], s_al[HQ_KV_MAX_REQUESTS + 1];
    __shared__ int32_t s_wave[2][kSlotThreads / 64];
    const int tid = threadIdx.x, B = (int)a.B;
#pragma unroll 4
    for (int r = tid; r < B; r += kSlotThreads) {
        const int32_t c = max(a.cached[r], 0), n = max(a.fresh[r], 0), kv = sat_add(c, n);
        s_c[r] = c;
        s_cu[r] = n;
        s_al[r] = pages_of(a.per_block, kv) - pages_of(a.per_block, c);
        if (blockIdx.x == 0) a.kv_lens[r] = kv;
    }
    __syncthreads();
    const int per = (B + kSlotThreads - 1) / kSlotThreads;  // consecutive requests of a thread
    const int r0 = min(tid * per, B), r1 = min(r0 + per, B);
    int32_t sum_n = 0, sum_p = 0;
    for (int r = r0; r < r1; ++r) {
        const int32_t n = s_cu[r], p = s_al[r];
        s_cu[r] = sum_n;
        s_al[r] = sum_p;
        sum_n = sat_add(sum_n, n);
        sum_p = sat_add(sum_p, p);
    }
    int32_t in_n = sum_n, in_p = sum_p;  // inclusive sums over the wave's threads
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t un = __shfl_up(in_n, off), up = __shfl_up(in_p, off);
        if ((tid & 63) >= off) {
            in_n = sat_add(in_n, un);
            in_p = sat_add(in_p, up);
        }
    }
    if ((tid & 63) == 63) {
        s_wave[0][tid >> 6] = in_n;
        s_wave[1][tid >> 6] = in_p;
    }
    __syncthreads();
    int32_t base_n = 0, base_p = 0, all_n = 0, all_p = 0;
    for (int w = 0; w < kSlotThreads / 64; ++w) {
        if (w == (tid >> 6)) {
            base_n = all_n;
            base_p = all_p;
        }
        all_n = sat_add(all_n, s_wave[0][w]);
        all_p = sat_add(all_p, s_wave[1][w]);
    }
    // exclusive over the wave: the inclusive sum of the lane before
    const int32_t ex_n = __shfl_up(in_n, 1), ex_p = __shfl_up(in_p, 1);
    if (tid & 63) {
        base_n = sat_add(base_n, ex_n);
        base_p = sat_add(base_p, ex_p);
    }
    for (int r = r0; r < r1; ++r) {
        s_cu[r] = sat_add(s_cu[r], base_n);
        s_al[r] = sat_add(s_al[r], base_p);
    }
    if (tid == 0) {
        s_cu[B] = all_n;
        s_al[B] = all_p;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int r = tid; r <= B; r += kSlotThreads) a.cu[r] = s_cu[r];
        if (tid == 0) a.taken[0] = all_p;
    }
    const int64_t stride = (int64_t)gridDim.x * kSlotThreads;
    const int64_t start = (int64_t)blockIdx.x * kSlotThreads + tid;
    for (int64_t i = start; i < all_p; i += stride) {
        const int r = owner_of(s_al, B, (int32_t)i);
        const int64_t col = pages_of(a.per_block, s_c[r]) + (i - s_al[r]);
        if (col < a.max_blocks) a.table[(int64_t)r * a.max_blocks + col] = i < a.n_free ? a.free_blocks[i] : -1;
    }
    for (int64_t t = start; t < a.T_cap; t += stride) {
        int32_t pos_out = 0;
        int64_t slot = -1;
        if (t < all_n) {
            const int r = owner_of(s_cu, B, (int32_t)t);
            const int32_t pos = sat_add(s_c[r], (int32_t)t - s_cu[r]);
            const int64_t col = a.per_block.div(pos), have = pages_of(a.per_block, s_c[r]);
            int64_t page = -1;
            if (col < a.max_blocks) {
                if (col < have) {
                    page = a.table[(int64_t)r * a.max_blocks + col];
                } else {
                    const int64_t at = s_al[r] + (col - have);
                    page = at < a.n_free ? a.free_blocks[at] : -1;
                }
            }
            if (page >= 0) slot = page * a.block_size + (pos - col * a.block_size);
            pos_out = sat_add((int32_t)a.first_pos, pos);
        }
        a.positions[t] = pos_out;
        a.slots[t] = slot;
    }
}

hipError_t kv_slots_launch(const KvSlotsArgs& a) {
    int64_t wgs = cdiv(a.T_cap > a.B ? a.T_cap : a.B, 2 * kSlotThreads);
    if (wgs < 1) wgs = 1;
    if (wgs > 512) wgs = 512;
    hipLaunchKernelGGL(kv_slots_kernel, dim3((unsigned)wgs), dim3(kSlotThreads), 0, a.stream, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// rotary table
// ---------------------------------------------------------------------------

// A thread writes `run` consecutive positions of one pair: cos and sin of the
// first in 64 bits, then each next one by turning that by the pair's step, four
// 64-bit operations, whose error after 32 steps is still below 2^-46; rounded once
// to fp32.  The first's angle is position * (turns + rest) less the nearest whole
// number of turns, by fma, so that the product is not rounded before that is
// taken off: right to 2^-30 of a turn at the last position, 2^-46 at 131072.  A
// library cos and sin for each element was bound by arithmetic (131072 positions
// x 128 elements: 22 us); this is bound by the stores (11 to 12.6 us, 5.3 to 6.1
// TB/s; a large fill reaches 6.8).
__global__ __launch_bounds__(256) void rope_table_kernel(RopeTableArgs a, int run) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row0 = i / a.half * run;
    if (row0 >= a.count) return;
    const int d = (int)(i - row0 / run * a.half);
    const double pos = (double)(a.first + row0), turn = fma(pos, a.turns[d], -rint(pos * a.turns[d]));
    double c, s, cs, ss;
    sincospi(2.0 * fma(pos, a.rest[d], turn), &s, &c);
    sincospi(2.0 * a.turns[d], &ss, &cs);  // (fewer than half a turn: base > 1)
    const int64_t end = min(row0 + run, a.count);
    float* at = a.table + row0 * 2 * a.half + d;
    for (int64_t row = row0; row < end; ++row, at += 2 * a.half) {
        at[0] = (float)(c * a.gain);
        at[a.half] = (float)(s * a.gain);
        const double c1 = c * cs - s * ss;
        s = s * cs + c * ss;
        c = c1;
    }
}

hipError_t rope_table_launch(const RopeTableArgs& a) {
    // longer runs share the cost of their start, as long as there are waves to fill the card
    const int64_t total = a.count * a.half;
    int run = 32;
    while (run > 4 && total / run < 256 * 1024) run /= 2;
    const int64_t wgs = cdiv(cdiv(a.count, run) * a.half, 256);
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)wgs), dim3(256), 0, a.stream, a, run);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// rotation and cache write
// ---------------------------------------------------------------------------

// Eight consecutive 16-bit elements as floats, and back.
template <bool BF16>
__device__ __forceinline__ void unpack8(v4u u, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bits16_to_f32<BF16>((uint16_t)(u[i] & 0xFFFFu));
        f[2 * i + 1] = bits16_to_f32<BF16>((uint16_t)(u[i] >> 16));
    }
}
template <bool BF16>
__device__ __forceinline__ v4u pack8(const float (&f)[8]) {
    v4u u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        u[i] = (uint32_t)f32_to_16<BF16>(f[2 * i]) | ((uint32_t)f32_to_16<BF16>(f[2 * i + 1]) << 16);
    return u;
}

// E4M3 codes of x / scale: fp32 division, nearest even, saturating, NaN kept.
__device__ __forceinline__ uint2 e4m3x8(const float (&f)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = f[4 * h + i] / scale;
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(c[0], -448.f), 448.f), fminf(fmaxf(c[1], -448.f), 448.f), 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(c[2], -448.f), 448.f), fminf(fmaxf(c[3], -448.f), 448.f), p, true);
        w[h] = (uint32_t)p;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c[i] != c[i]) w[h] = (w[h] & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
    }
    return make_uint2(w[0], w[1]);
}

// A unit is 16 elements of one head: eight pairs of the rotated part, or 16
// elements that pass through; one thread each, all heads of a token side by side,
// so that q, k and v are read and written once in whole lines and the table's row
// comes from cache.  Bound by memory: 16384 tokens of 64 + 2 x 8 heads of 128 into
// an 8-bit cache 131 us, 4.9 TB/s (a large copy reaches 5.2).
template <bool BF16, bool FP8>
__global__ __launch_bounds__(256) void rope_kv_kernel(RopeKvArgs a) {
#pragma clang fp contract(off)
    const int64_t t = blockIdx.x;
    const int D16 = a.kv.head_dim / 16, hk = a.kv.kv_heads;
    const int units = (a.q_heads + 2 * hk) * D16;
    const int u = blockIdx.y * 256 + threadIdx.x;
    if (u >= units) return;
    const int head = u / D16, part = u - head * D16;
    const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + hk;
    const uint16_t* src;
    uint16_t* dst = nullptr;
    uint8_t* dst8 = nullptr;
    float scale = 1.f;
    bool store = true;
    if (is_q) {
        src = (const uint16_t*)a.q + t * a.q_stride + (int64_t)head * a.kv.head_dim;
        dst = (uint16_t*)a.q_out + t * a.q_out_stride + (int64_t)head * a.kv.head_dim;
    } else {
        const int h = is_v ? head - a.q_heads - hk : head - a.q_heads;
        src = is_v ? (const uint16_t*)a.v + t * a.v_stride : (const uint16_t*)a.k + t * a.k_stride;
        src += (int64_t)h * a.kv.head_dim;
        const int64_t slot = a.slots[t];
        store = slot >= 0 && slot < a.kv.num_blocks * a.kv.block_size;
        const uint32_t page = store ? a.kv.per_block.div((uint32_t)slot) : 0u;
        const int64_t off = (int64_t)page * a.kv.block_stride + (int64_t)((store ? (uint32_t)slot : 0u) - page * (uint32_t)a.kv.block_size) * a.kv.slot_stride +
                            (int64_t)h * a.kv.head_stride;
        void* base = is_v ? a.v_cache : a.k_cache;
        if constexpr (FP8) {
            dst8 = (uint8_t*)base + off;
            scale = (is_v ? a.v_scale : a.k_scale)[h];
        } else {
            dst = (uint16_t*)base + off;
        }
    }
    const bool turn = !is_v && 16 * part < a.rot;
    const int half = a.rot / 2;
    // element offsets of the unit's two groups of eight
    const int e0 = turn && !a.interleaved ? 8 * part : 16 * part;
    const int e1 = turn && !a.interleaved ? half + 8 * part : 16 * part + 8;
    float x[8], y[8];
    unpack8<BF16>(ld16(src + e0), x);
    unpack8<BF16>(ld16(src + e1), y);
    if (turn) {
        int64_t pos = a.positions[t];
        pos = pos < 0 ? 0 : pos >= a.table_rows ? a.table_rows - 1 : pos;
        const float* row = a.table + pos * a.rot + 8 * part;
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const v4f c = *(const v4f*)(row + 4 * i), s = *(const v4f*)(row + half + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cs[4 * i + j] = c[j];
                sn[4 * i + j] = s[j];
            }
        }
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p0 = x[2 * i], p1 = x[2 * i + 1], r0 = y[2 * i], r1 = y[2 * i + 1];
                x[2 * i] = p0 * cs[i] - p1 * sn[i];
                x[2 * i + 1] = p1 * cs[i] + p0 * sn[i];
                y[2 * i] = r0 * cs[4 + i] - r1 * sn[4 + i];
                y[2 * i + 1] = r1 * cs[4 + i] + r0 * sn[4 + i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p0 = x[i], p1 = y[i];
                x[i] = p0 * cs[i] - p1 * sn[i];
                y[i] = p1 * cs[i] + p0 * sn[i];
            }
        }
    }
    if (!store) return;
    if (FP8 && !is_q) {
        *(uint2*)(dst8 + e0) = e4m3x8(x, scale);
        *(uint2*)(dst8 + e1) = e4m3x8(y, scale);
    } else {
        *(v4u*)(dst + e0) = pack8<BF16>(x);
        *(v4u*)(dst + e1) = pack8<BF16>(y);
    }
}

hipError_t rope_kv_launch(const RopeKvArgs& a) {
    const int units = (a.q_heads + 2 * a.kv.kv_heads) * (a.kv.head_dim / 16);
    const dim3 grid((unsigned)a.T, (unsigned)cdiv(units, 256)), blk(256);
    const bool fp8 = a.kv.dtype == HQ_DT_FP8_E4M3;
    if (a.bf16 && fp8) hipLaunchKernelGGL((rope_kv_kernel<true, true>), grid, blk, 0, a.stream, a);
    else if (a.bf16) hipLaunchKernelGGL((rope_kv_kernel<true, false>), grid, blk, 0, a.stream, a);
    else if (fp8) hipLaunchKernelGGL((rope_kv_kernel<false, true>), grid, blk, 0, a.stream, a);
    else hipLaunchKernelGGL((rope_kv_kernel<false, false>), grid, blk, 0, a.stream, a);
    return hipGetLastError();
}

}  // namespace hq
