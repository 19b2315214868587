// Internal interface of the operators around (and with) the 8-bit expert
// products of a mixture-of-experts layer: norm and SwiGLU with quantised
// output, routing, FP8 experts, the weighted sum.  Arguments are checked by
// hq_api.cpp; launched by k_norm.hip, k_route.hip and k_moe_f8.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/hq.h"

namespace hq {

// What a row kernel writes: 16 bits, or codes with their scales.
enum class RowOut { SAME16, TOKEN_F8, TOKEN_I8, BLOCK_F8, MX_F8, MX_F4 };

struct RowArgs {
    bool silu;  // SwiGLU of [rows][2 width], else the norm
    bool bf16, w_f32;
    RowOut kind;
    int64_t rows;
    int width;
    float eps, w_offset;
    const void *x, *res, *w;
    int64_t x_stride, res_stride, sum_stride;
    void *sum, *out, *scale;
    hipStream_t stream;
};
hipError_t row_launch(const RowArgs& a);
constexpr int kRowMaxWidth = 65536;  // the longest row that a workgroup holds in registers

struct RouteArgs {
    int dtype, experts, top_k, groups, top_groups, group_best;
    bool sigmoid, renorm;
    float scale;
    int64_t T, stride;
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    hipStream_t stream;
};
hipError_t route_launch(const RouteArgs& a);
constexpr int kRouteMaxTopK = 64, kRouteMaxGroups = 64, kRouteMaxExperts = 4096;

struct CombineArgs {
    bool bf16;
    int64_t T, N;
    int top_k;
    const void *y, *add;
    const float* weights;
    const int32_t* sorted;
    void* out;
    int32_t* place;  // [T * top_k], with `sorted`
    hipStream_t stream;
};
hipError_t combine_launch(const CombineArgs& a);

// out[i] = A[sorted[i] / top_k], rows of `words` 32-bit words
hipError_t gather_words_launch(const void* A, const int* sorted, int64_t P, int top_k, int64_t words, void* out, hipStream_t st);

struct MoeF8Args {
    int64_t T, N, K;
    int top_k, E;
    bool indexed;
    const void* A;
    const float* sa;
    const int *ids, *offsets;
    const void *w, *s;
    void* D;
    void* ws;
    hipStream_t stream;
};
size_t moe_f8_workspace(int64_t T, int top_k, int E);
hipError_t moe_f8_launch(const MoeF8Args& a);

}  // namespace hq
