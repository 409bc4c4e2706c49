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
// from the lane rot_dim / 16 away (four dwords of raw input).
//
// With many tokens a wave takes one token and goes over its heads: the
// cosines, sines and norm weights, six times a row's own bytes, are then read
// once a wave and stay in registers.  With few it takes the rows that it
// holds at once, which spreads a token over the chip.  Rows / tokens, us, 32
// query and 8 key heads of 128, norm and full rotation: 64 tokens 3.0 / 8.4,
// 512 4.6 / 8.8, 2000 12.3 / 12.9, 4000 20.4 / 17.4, 16384 98 / 70 (4.8 TB/s,
// what a copy of as many bytes reaches).
#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4; // rows of a token a lane asks for before it works on the first (2: the same)
constexpr int64_t kMaxBlocks = 1 << 22; // a launch has fewer than 2^32 threads

// A row for every head_dim / 8 lanes.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void rope_rows_kernel(NormRopeArgs a)
{
    constexpr int LPR = D / 8; // lanes a row
    const int lane = __lane_id();
    const int l = lane & (LPR - 1);
    const uint32_t heads = (uint32_t)(a.q_heads + a.kv_heads);
    const uint32_t row = (blockIdx.x * kThreads + threadIdx.x) / LPR;
    const uint32_t token = row / heads, head = row - token * heads;
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

// What a wave keeps while it goes over heads: out_e = inv * (x_e cos_e g_e +
// y_e sin_e g'_e), with y the pair's other channel.
template <int D>
struct Turn {
    float c[8], s[8]; // of this lane's channels; the sign of the pair in s
    uint32_t keep;    // all ones where the lane's channels turn, else 0
    int from;         // byte index of the lane that holds the other channels
    bool pairs;
};

template <int DT, int D, bool NORM>
__device__ __forceinline__ void turn_heads(const uint16_t *src, uint16_t *dst, int first, int step, int heads, const uint16_t *weight,
                                           float eps, const Turn<D> &turn)
{
    constexpr int LPR = D / 8; // lanes a row
    const int l = __lane_id() & (LPR - 1);
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        c[e] = turn.c[e];
        s[e] = turn.s[e];
    }
    if (NORM) {
        const u32x4_t own = *reinterpret_cast<const u32x4_t *>(weight + l * 8);
        u32x4_t far;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            far[i] = turn.pairs ? __builtin_amdgcn_alignbit(own[i], own[i], 16)
                                : (uint32_t)__builtin_amdgcn_ds_bpermute(turn.from, (int)own[i]);
        float g[8], h[8];
        unpack8<DT>(own, g);
        unpack8<DT>(far, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] *= g[e];
            s[e] = turn.keep ? s[e] * h[e] : 0.0f;
        }
    }
    for (int base = first; base < heads; base += kBatch * step) {
        u32x4_t raw[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int head = base + b * step;
            if (b == 0 || head < heads)
                raw[b] = *reinterpret_cast<const u32x4_t *>(src + (int64_t)head * D + l * 8);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int head = base + b * step;
            if (b > 0 && !__any(head < heads))
                break;
            float x[8], y[8], inv = 1.0f;
            unpack8<DT>(raw[b], x);
            if (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss += x[e] * x[e];
#pragma unroll
                for (int d = 1; d < LPR; d <<= 1)
                    ss += shfl_xor_f32(ss, d);
                inv = 1.0f / sqrtf(ss * (1.0f / D) + eps);
            }
            u32x4_t other;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                other[i] = (turn.pairs ? __builtin_amdgcn_alignbit(raw[b][i], raw[b][i], 16)
                                       : (uint32_t)__builtin_amdgcn_ds_bpermute(turn.from, (int)raw[b][i])) &
                           turn.keep; // (what does not turn must not meet an infinity times 0)
            unpack8<DT>(other, y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = fmaf(x[e] * inv, c[e], y[e] * inv * s[e]);
            if (head < heads)
                *reinterpret_cast<u32x4_t *>(dst + (int64_t)head * D + l * 8) = pack8<DT>(x);
        }
    }
}

// A token for every wave.
template <int DT, int D, bool NORM>
__device__ __forceinline__ void turn_token(const NormRopeArgs &a, int64_t token)
{
    constexpr int LPR = D / 8, RPW = 64 / LPR; // rows a wave holds
    const int lane = __lane_id(), l = lane & (LPR - 1), first = lane / LPR;
    const int32_t pos = a.positions[token];
    const uint16_t *q = a.q + token * a.q_stride, *k = a.k + token * a.k_stride;
    uint16_t *q_out = a.q_out + token * a.q_out_stride, *k_out = a.k_out + token * a.k_out_stride;
    if (pos < 0 || pos >= a.max_position) {
        for (int h = first; h < a.q_heads; h += RPW)
            *reinterpret_cast<u32x4_t *>(q_out + (int64_t)h * D + l * 8) = (u32x4_t){0, 0, 0, 0};
        for (int h = first; h < a.kv_heads; h += RPW)
            *reinterpret_cast<u32x4_t *>(k_out + (int64_t)h * D + l * 8) = (u32x4_t){0, 0, 0, 0};
        return;
    }
    const int half = a.rot_dim / 2, d0 = l * 8;
    const bool turns = d0 < a.rot_dim, low = d0 < half;
    Turn<D> turn;
    turn.pairs = a.interleaved;
    turn.keep = turns ? ~0u : 0u;
    turn.from = (lane - l + ((low ? l + half / 8 : l - half / 8) & (LPR - 1))) << 2;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        turn.c[e] = 1.0f;
        turn.s[e] = 0.0f;
    }
    if (turns) {
        const int at = a.interleaved ? d0 / 2 : (low ? d0 : d0 - half);
        const float *cos = a.cos + (int64_t)pos * half + at, *sin = a.sin + (int64_t)pos * half + at;
        if (a.interleaved) {
            const float4_t c = *reinterpret_cast<const float4_t *>(cos), s = *reinterpret_cast<const float4_t *>(sin);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                turn.c[e] = c[e / 2];
                turn.s[e] = e & 1 ? s[e / 2] : -s[e / 2];
            }
        } else {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4_t c = *reinterpret_cast<const float4_t *>(cos + 4 * v), s = *reinterpret_cast<const float4_t *>(sin + 4 * v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    turn.c[4 * v + e] = c[e];
                    turn.s[4 * v + e] = low ? -s[e] : s[e];
                }
            }
        }
    }
    turn_heads<DT, D, NORM>(q, q_out, first, RPW, a.q_heads, a.q_weight, a.eps, turn);
    turn_heads<DT, D, NORM>(k, k_out, first, RPW, a.kv_heads, a.k_weight, a.eps, turn);
}

template <int DT, int D, bool NORM>
__global__ __launch_bounds__(kThreads) void rope_tokens_kernel(NormRopeArgs a)
{
    const uint32_t waves = gridDim.x * (kThreads / 64);
    for (int64_t token = blockIdx.x * (kThreads / 64) + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
         token < a.tokens; token += waves)
        turn_token<DT, D, NORM>(a, token);
}

template <int DT, int D>
hipError_t launch(const NormRopeArgs &a, hipStream_t stream)
{
    // A wave a token from where these are the four waves that a SIMD holds.
    const int64_t lanes = a.tokens * (a.q_heads + a.kv_heads) * (D / 8);
    const dim3 block(kThreads);
    if (a.tokens < 16 * (int64_t)device_cu_count() && lanes < int64_t(1) << 31) {
        rope_rows_kernel<DT, D><<<dim3((unsigned)((lanes + kThreads - 1) / kThreads)), block, 0, stream>>>(a);
        return hipGetLastError();
    }
    const int64_t blocks = (a.tokens + kThreads / 64 - 1) / (kThreads / 64);
    const dim3 grid((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
    if (a.q_weight)
        rope_tokens_kernel<DT, D, true><<<grid, block, 0, stream>>>(a);
    else
        rope_tokens_kernel<DT, D, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_type(const NormRopeArgs &a, hipStream_t stream)
{
    return a.head_dim == 64 ? launch<DT, 64>(a, stream) : a.head_dim == 128 ? launch<DT, 128>(a, stream) : hipErrorInvalidValue;
}

} // namespace

hipError_t launch_qk_norm_rope(const NormRopeArgs &a, int dtype, hipStream_t stream)
{
    return dtype == QW_F16 ? launch_type<QW_F16>(a, stream) : launch_type<QW_BF16>(a, stream);
}

} // namespace qw
