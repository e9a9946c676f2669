// E4M3 storage of activations: loads and the 1 x 128 block of 16 lanes.
#pragma once

#include "tq_dense.cuh"

#include <type_traits>

namespace tq {

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value) f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// One 128-wide block held by 16 consecutive lanes, 8 values each (both halves of the warp
// call it): the lane's E4M3 bytes, and the block's scale.
__device__ __forceinline__ uint2 fp8_store_block(const float (&v)[8], float &scale) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = finite_max(m, v[j]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = e4m3_block_exponent(m);
    const float inv = exp2_int(-e);
    scale = exp2_int(e);
    return make_uint2(e4m3x4_scaled(v[0], v[1], v[2], v[3], inv), e4m3x4_scaled(v[4], v[5], v[6], v[7], inv));
}

}  // namespace tq
