// qk_norm_rope.hip -- RMS norm of each query and key head, and the rotation
// by position, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (w null: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   for the pairs of
//   the first rot_dim channels: (2 i, 2 i + 1), or (i, i + rot_dim / 2)
//
// in fp32, rounded once to the 16-bit output type.
//
// Bound by HBM: each element is read once and written once, 2 bytes each.
// A row (token, head) is held by head_dim / 8 lanes, 16 bytes a lane, so a
// wave reads and writes whole contiguous rows; the row's sum of squares is
// a butterfly over those lanes, and the far half of a half-split pair comes
// from the lane rot_dim / 16 away (four dwords of raw input; its norm
// weight is read again, from cache).
#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

namespace {

constexpr int kThreads = 256;

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(NormRopeArgs a)
{
    constexpr int LPR = D / 8; // lanes a row
    const int lane = __lane_id();
    const int l = lane & (LPR - 1);
    const uint32_t heads = (uint32_t)(a.q_heads + a.kv_heads);
    const uint64_t row = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / LPR;
    const uint32_t token = (uint32_t)(row / heads);
    const uint32_t head = (uint32_t)(row % heads);
    if (token >= a.tokens)
        return; // whole rows of LPR lanes leave together; shuffles stay within a row
    const bool is_q = head < (uint32_t)a.q_heads;
    const uint32_t h = is_q ? head : head - (uint32_t)a.q_heads;
    const uint16_t *src = (is_q ? a.q + (int64_t)token * a.q_stride : a.k + (int64_t)token * a.k_stride) + h * D + l * 8;
    uint16_t *dst = (is_q ? a.q_out + (int64_t)token * a.q_out_stride : a.k_out + (int64_t)token * a.k_out_stride) +
                    h * D + l * 8;
    const int32_t pos = a.positions[token];
    if (pos < 0 || pos >= a.max_position) {
        *reinterpret_cast<u32x4_t *>(dst) = (u32x4_t){0, 0, 0, 0};
        return;
    }
    const u32x4_t raw = *reinterpret_cast<const u32x4_t *>(src);
    float x[8];
    unpack8<DT>(raw, x);
    const uint16_t *w = is_q ? a.q_weight : a.k_weight;
    float inv = 1.0f;
    if (w) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss += x[i] * x[i];
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1)
            ss += shfl_xor_f32(ss, d);
        inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
        float g[8];
        unpack8<DT>(*reinterpret_cast<const u32x4_t *>(w + l * 8), g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = x[i] * inv * g[i];
    }
    const int half = a.rot_dim / 2;
    const int d0 = l * 8;
    if (a.interleaved) {
        if (d0 < a.rot_dim) {
            const float4_t c = *reinterpret_cast<const float4_t *>(a.cos + (int64_t)pos * half + d0 / 2);
            const float4_t s = *reinterpret_cast<const float4_t *>(a.sin + (int64_t)pos * half + d0 / 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i], v = x[2 * i + 1];
                x[2 * i] = u * c[i] - v * s[i];
                x[2 * i + 1] = v * c[i] + u * s[i];
            }
        }
    } else {
        const int step = half / 8;
        const bool low = d0 < half;
        const int partner = low ? l + step : l - step;
        const int from = (lane - l + (partner & (LPR - 1))) << 2;
        u32x4_t other;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            other[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)raw[i]);
        if (d0 < a.rot_dim) {
            float y[8];
            unpack8<DT>(other, y);
            if (w) {
                float g[8];
                unpack8<DT>(*reinterpret_cast<const u32x4_t *>(w + partner * 8), g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = y[i] * inv * g[i];
            }
            const int at = low ? d0 : d0 - half;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4_t c = *reinterpret_cast<const float4_t *>(a.cos + (int64_t)pos * half + at + 4 * v);
                const float4_t s = *reinterpret_cast<const float4_t *>(a.sin + (int64_t)pos * half + at + 4 * v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float t = y[4 * v + i] * s[i];
                    x[4 * v + i] = x[4 * v + i] * c[i] + (low ? -t : t);
                }
            }
        }
    }
    *reinterpret_cast<u32x4_t *>(dst) = pack8<DT>(x);
}

template <int DT>
hipError_t launch(const NormRopeArgs &a, hipStream_t stream)
{
    const uint64_t lanes = (uint64_t)a.tokens * (uint64_t)(a.q_heads + a.kv_heads) * (uint64_t)(a.head_dim / 8);
    const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads)), block(kThreads);
    switch (a.head_dim) {
    case 64:
        qk_norm_rope_kernel<DT, 64><<<grid, block, 0, stream>>>(a);
        break;
    case 128:
        qk_norm_rope_kernel<DT, 128><<<grid, block, 0, stream>>>(a);
        break;
    default:
        return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

} // namespace

hipError_t launch_qk_norm_rope(const NormRopeArgs &a, int dtype, hipStream_t stream)
{
    return dtype == QW_F16 ? launch<QW_F16>(a, stream) : launch<QW_BF16>(a, stream);
}

} // namespace qw
