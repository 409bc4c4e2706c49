// kv_device.h -- device helpers of the paged KV cache kernels: the two
// 16-bit activation types and cross-lane reductions on whole wavefronts.
#pragma once

#include "qw.h"
#include "qw_device.h"

namespace qw {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float float16_t __attribute__((ext_vector_type(16)));

// A 16-bit activation type by its qw_dtype code.
template <int DT>
struct Act;
template <>
struct Act<QW_F16> {
    static __device__ __forceinline__ float lo(uint32_t v) { return (float)as_half2(v).x; }
    static __device__ __forceinline__ float hi(uint32_t v) { return (float)as_half2(v).y; }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const half2_t h = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, h);
    }
};
template <>
struct Act<QW_BF16> {
    static __device__ __forceinline__ float lo(uint32_t v) { return __builtin_bit_cast(float, v << 16); }
    static __device__ __forceinline__ float hi(uint32_t v) { return __builtin_bit_cast(float, v & 0xffff0000u); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const bf16x2_t h = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, h);
    }
};

template <int DT>
__device__ __forceinline__ void unpack8(const u32x4_t v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = Act<DT>::lo(w[i]);
        f[2 * i + 1] = Act<DT>::hi(w[i]);
    }
}

template <int DT>
__device__ __forceinline__ u32x4_t pack8(const float (&f)[8])
{
    return (u32x4_t){Act<DT>::pack(f[0], f[1]), Act<DT>::pack(f[2], f[3]), Act<DT>::pack(f[4], f[5]),
                     Act<DT>::pack(f[6], f[7])};
}

// Reductions over lanes l, l ^ 16 and l, l ^ 32 by the gfx950 row swaps
// (plain VALU operations; a trip through the LDS crossbar would cost its
// latency in the inner loop).
__device__ __forceinline__ float max_xor32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float max_xor16(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float add_xor32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float add_xor16(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

__device__ __forceinline__ float wave_max_f32(float v)
{
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1)
        v = fmaxf(v, shfl_xor_f32(v, d));
    return max_xor32(max_xor16(v));
}

__device__ __forceinline__ int64_t shfl_up_i64(int64_t v, int d)
{
    const int src = (int)__lane_id() - d;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(src << 2, (int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_bpermute(src << 2, (int)(uint32_t)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

} // namespace qw
