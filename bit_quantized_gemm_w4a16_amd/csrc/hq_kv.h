// Internal interface of the paged key/value cache operators (slot maps, rotary
// positions, attention): arguments checked by hq_api.cpp, launched by k_kv.hip
// and k_attn.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/hq.h"

namespace hq {

// Division of n in 0 .. 2^31-1 by a constant d >= 1 as one high multiply:
// with 2^(s-1) < d <= 2^s and m = floor(2^(31+s) / d) + 1, m d exceeds 2^(31+s)
// by at most d <= 2^s, so floor(n m / 2^(31+s)) = floor(n / d) for n < 2^31.
// m needs at most 32 bits except at d = 1, which has its own flag.
struct FastDiv {
    uint32_t d, m, s;  // s: shift after the high multiply (31 + s - 32)
    static FastDiv of(uint32_t d) {
        FastDiv f{d, 0, 0};
        if (d == 1) return f;
        uint32_t s = 0;
        while (((uint64_t)1 << s) < d) ++s;
        f.m = (uint32_t)((((uint64_t)1 << (31 + s)) / d) + 1);
        f.s = s - 1;
        return f;
    }
    __host__ __device__ uint32_t div(uint32_t n) const {
        return m == 0 ? n : (uint32_t)(((uint64_t)n * m) >> 32) >> s;
    }
};

// A cache as the kernels see it.
struct KvLayout {
    int64_t block_stride, slot_stride, head_stride;  // elements
    int64_t num_blocks;
    int kv_heads, head_dim, block_size;
    FastDiv per_block;
    int dtype;  // hq_dtype
};

struct KvSlotsArgs {
    int block_size;
    FastDiv per_block;
    int64_t B, T_cap, max_blocks, first_pos, n_free;
    const int32_t *cached, *fresh, *free_blocks;
    int32_t *table, *cu, *kv_lens, *positions, *taken;
    int64_t* slots;
    hipStream_t stream;
};
hipError_t kv_slots_launch(const KvSlotsArgs& a);

struct RopeTableArgs {
    double turns[128], rest[128];  // turns of one position step, per pair, in two parts
    double gain;
    int64_t first, count;
    int half;
    float* table;
    hipStream_t stream;
};
hipError_t rope_table_launch(const RopeTableArgs& a);

struct RopeKvArgs {
    KvLayout kv;
    bool bf16, interleaved;
    int rot, q_heads;
    int64_t T, q_stride, k_stride, v_stride, q_out_stride, table_rows;
    const void *q, *k, *v;
    const int32_t* positions;
    const float* table;
    const int64_t* slots;
    void *q_out, *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    hipStream_t stream;
};
hipError_t rope_kv_launch(const RopeKvArgs& a);

struct AttnArgs {
    KvLayout kv;
    bool bf16;
    int q_heads;
    int64_t B, T, q_stride, out_stride, prefix_len, max_blocks;
    int64_t max_new, max_kv, total_kv;
    float scale, softcap;
    const void *q, *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *prefix_table, *block_table, *kv_lens, *cu;
    void* out;
    float* lse;
    void* ws;
    hipStream_t stream;
};
size_t attn_workspace(const AttnArgs& a);   // host only, reads the sizes; SIZE_MAX: more workgroups than one launch holds
hipError_t attn_launch(const AttnArgs& a);  // records the launches instead while a PlanRecorder is active

}  // namespace hq
