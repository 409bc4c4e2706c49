// epilogue_device.h -- what the products' epilogues share: activations, the
// 16-bit output types, and which rows a workgroup of a grouped product takes.
#pragma once

#include "qw_device.h"
#include "qw_internal.h"

namespace qw {

// v / (1 + exp(-z)): silu for z = v.  exp(-z) may overflow to infinity, which
// gives the limit 0.
__device__ __forceinline__ float times_sigmoid(float v, float z)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// v Phi(v), Phi the normal distribution function.  For z = |v|,
// Phi(-z) = exp(-z^2 / 2) t P(t) with t = 1 / (1 + z / 4): P is a least
// squares fit of erfcx(z / sqrt 2) / (2 t), reweighted towards equal relative
// errors; in fp32 the product is off by at most 1.9e-6 relative for z < 6.
__device__ __forceinline__ float gelu(float v)
{
    const float z = fabsf(v);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.25f, z, 1.0f));
    float p = -0.039373025f;
    p = fmaf(p, t, 0.0861854f);
    p = fmaf(p, t, 0.006413045f);
    p = fmaf(p, t, 0.07401459f);
    p = fmaf(p, t, 0.07976867f);
    p = fmaf(p, t, 0.093513884f);
    p = fmaf(p, t, 0.09974142f);
    p = fmaf(p, t, 0.09973546f);
    const float tail = p * t * __expf(-0.5f * z * z);
    return v * (v < 0.0f ? tail : 1.0f - tail);
}

// v (1 + tanh(u)) / 2 = v / (1 + exp(-2 u)), u = sqrt(2 / pi) (v + 0.044715 v^3)
__device__ __forceinline__ float gelu_tanh(float v)
{
    return times_sigmoid(v, v * fmaf(0.0713548163f, v * v, 1.59576912f));
}

__device__ __forceinline__ float relu(float v) { return v < 0.0f ? 0.0f : v; } // (keeps a NaN)

__device__ __forceinline__ float activate(int activation, float v)
{
    switch (activation) {
    case QW_ACT_RELU:
        return relu(v);
    case QW_ACT_GELU:
        return gelu(v);
    case QW_ACT_GELU_TANH:
        return gelu_tanh(v);
    case QW_ACT_SILU:
        return times_sigmoid(v, v);
    default:
        return v;
    }
}

__device__ __forceinline__ float from16(uint16_t b, int bf16)
{
    return bf16 ? __builtin_bit_cast(float, (uint32_t)b << 16) : f16_bits_to_f32(b);
}

// Rounds to nearest even, either way.
__device__ __forceinline__ uint16_t to16(float v, int bf16)
{
    return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)v) : f32_to_f16_bits(v);
}

// ---------------------------------------------------------------------------
// Row tiles of a grouped product.  With o_e the first entry of expert e, its
// tiles of B rows begin at number floor(o_e / B) + e: the next expert's begin
// floor(o_{e+1} / B) - floor(o_e / B) + 1 further on, which is at least the
// ceil((o_{e+1} - o_e) / B) tiles it has.  So no sums over experts are needed
// to lay the tiles out, and floor(entries / B) + count + 1 numbers hold them
// all, those of the entries behind the last expert's (number `count` here)
// among them.  A number beyond its expert's tiles has nothing to do.
// ---------------------------------------------------------------------------
struct GroupTile {
    int expert; // `count`: entries of no expert
    int begin, end;
};

// All 64 lanes take part; the result is uniform.  Offsets are taken as within
// [0, entries], so that no tile lies outside; `end` <= `begin`: nothing to do.
template <int B>
__device__ __forceinline__ GroupTile group_tile(const Experts &ex, int tile)
{
    const int lane = __lane_id();
    int upto = 0; // experts that begin at or before this tile (offsets do not decrease)
    for (int base = 0; base <= ex.count; base += kWave) {
        const int e = base + lane;
        const int o = e <= ex.count ? min(max(ex.offsets[e], 0), ex.entries) : 0;
        upto += __popcll(__ballot(e <= ex.count && o / B + e <= tile));
    }
    GroupTile g = {upto - 1, 0, 0};
    if (upto > 0) {
        const int lo = min(max(ex.offsets[upto - 1], 0), ex.entries);
        const int hi = upto <= ex.count ? min(max(ex.offsets[upto], 0), ex.entries) : ex.entries;
        const int64_t first = lo + (int64_t)(tile - lo / B - (upto - 1)) * B;
        if (first >= lo && first < hi) { // (below lo only where offsets decrease)
            g.begin = (int)first;
            g.end = hi;
        }
    }
    return g;
}

// Activation row of entry p, or -1 where its index is not one.
__device__ __forceinline__ int entry_row(const Experts &ex, int p)
{
    if (!ex.rows)
        return p;
    const int flat = ex.rows[p];
    const int row = flat / ex.top_k;
    return flat >= 0 && row < ex.x_rows ? row : -1;
}

} // namespace qw
