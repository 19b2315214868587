// Rows of 16-bit elements in groups of eight, for the operators of a routed layer.
#pragma once
#include "hq_device.hpp"

namespace hq {

namespace {

template <bool BF16>
__device__ __forceinline__ void unpack8(v4u v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = v[i];
        f[2 * i] = bits16_to_f32<BF16>((uint16_t)u);
        f[2 * i + 1] = bits16_to_f32<BF16>((uint16_t)(u >> 16));
    }
}
template <bool BF16>
__device__ __forceinline__ v4u pack8(const float (&f)[8]) {
    v4u v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (uint32_t)f32_to_16<BF16>(f[2 * i]) | ((uint32_t)f32_to_16<BF16>(f[2 * i + 1]) << 16);
    return v;
}

// Eight 16-bit elements at `at`, of which n are the row's (the others read as 0).  VEC: the
// address is a multiple of 16 and n is 8 or less than 1.  Without it rows start at any element: the
// same wide access, which the memory takes at any alignment, and the row's last group by
// elements.  NT: past the caches.
typedef v4u v4u_any __attribute__((aligned(2)));
template <bool VEC, bool NT = false>
__device__ __forceinline__ v4u load8(const uint16_t* at, int n) {
    if (n >= 8) {
        if constexpr (NT) return VEC ? ld_nt((const v4u*)at) : __builtin_nontemporal_load((const v4u_any*)at);
        else return VEC ? ld16(at) : *(const v4u_any*)at;
    }
    v4u v{0, 0, 0, 0};
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) v[i >> 1] |= (uint32_t)at[i] << (16 * (i & 1));
    }
    return v;
}
template <bool VEC>
__device__ __forceinline__ void store8(uint16_t* at, v4u v, int n) {
    if (n >= 8) {
        if constexpr (VEC) *(v4u*)at = v;
        else *(v4u_any*)at = v;
    } else if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) at[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
}

}  // namespace

}  // namespace hq
