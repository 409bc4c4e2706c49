// kv_attention_device.h -- what the attention kernels over the paged KV cache
// share: a request's sizes as the device holds them, and query rows as fp16
// operands.
#pragma once

#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

// The weights P = 2^{t - M} are rounded to fp16 for the second product: by
// 2^-11 of a weight from 2^-14 on, by 2^-25 below, where fp16 is subnormal.
// So a reference M is set kKvRise below the row's largest exponent t: the largest
// weight is 2^8 then, weights down to 2^-22 of it keep all bits, and only those
// below 2^-33 of it are in the denominator alone (with the largest at 1: 2^-25,
// which the keys of a long context behind one dominant key reach: lost, with all
// that such a row gives).  A reference moves where the weights of 8 or 16 keys of a lane add up to
// kKvLarge, fp16's largest number, below which none of them overflows; they move
// more often the higher the rise: 0, 8 and 10: 292, 295 and 297 us for three
// prompts of up to 4096 tokens, 554, 560 and 568 for eight chunks of 512 behind
// 15000.  A maximum above kKvNothing is one of scores, not of masked places.
constexpr float kKvRise = 8.0f, kKvLarge = 65504.0f, kKvNothing = -3e38f;

__device__ __forceinline__ int kv_clamp(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// What one request asks for, bounded by what the arguments describe.
struct KvRequest {
    int t0, past; // first token; cached tokens before it (negative where there are more queries than cached tokens)
    int ctx;      // cached tokens
    int rows;     // query rows of a key head: those of at most max_new tokens; 0 if the launch does not take them
};

__device__ __forceinline__ KvRequest kv_request(const KvAttnArgs &a, int r)
{
    KvRequest s;
    s.t0 = kv_clamp(a.cu_tokens[r], 0, a.tokens);
    const int n = kv_clamp(a.cu_tokens[r + 1], s.t0, a.tokens) - s.t0;
    s.ctx = kv_clamp(a.context[r], 0, a.max_context);
    s.past = s.ctx - n;
    const int rows = (n < a.max_new ? n : a.max_new) * a.group;
    s.rows = rows >= a.least_rows && rows <= a.most_rows ? rows : 0;
    return s;
}

// The tokens of no request, as one without keys: those behind the last one's
// (g = 0), and before the first one's (g = 1).
__device__ __forceinline__ KvRequest kv_gap(const KvAttnArgs &a, int g)
{
    const int edge = kv_clamp(a.cu_tokens[g ? 0 : a.requests], 0, a.tokens), n = g ? edge : a.tokens - edge;
    return {g ? 0 : edge, -n, 0, n * a.group};
}

// Row block number `target` of all requests' in a row, `per` rows a block: its
// request and its number in it, or false behind the last one.  Within a request
// the last rows come first: under a causal mask they have the most keys.  For
// workgroups of 64 NW threads; `sums` and `found` are theirs, free to use.
template <int NW, typename Rows>
__device__ __forceinline__ bool kv_find_block(int requests, int per, Rows rows_of, int target, int *sums, int *found, int &request,
                                              int &block)
{
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    for (int base = 0;; base += 64 * NW) {
        if (base >= requests)
            return false;
        const int mine = base + (int)threadIdx.x;
        const int rows = rows_of(mine < requests ? mine : requests - 1);
        const int blocks = mine < requests ? (rows + per - 1) / per : 0;
        int upto = blocks;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(upto, d);
            upto += lane >= d ? up : 0;
        }
        if (lane == 63)
            sums[wave] = upto;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            upto += w < wave ? sums[w] : 0;
            total += sums[w];
        }
        if (target < upto && target >= upto - blocks) {
            found[0] = mine;
            found[1] = upto - 1 - target;
        }
        __syncthreads();
        if (target < total)
            break;
        target -= total;
    }
    request = __builtin_amdgcn_readfirstlane(found[0]);
    block = __builtin_amdgcn_readfirstlane(found[1]);
    return true;
}

// 8 activations -> fp16 (bf16 after multiplication by `up`, a power of two).
template <int DT>
__device__ __forceinline__ half8_t kv_half8(u32x4_t v, float up)
{
    if (DT == QW_F16)
        return __builtin_bit_cast(half8_t, v);
    float f[8];
    unpack8<DT>(v, f);
    half8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h[i] = (_Float16)(f[i] * up);
    return h;
}

// The power of two that brings a bf16 row's largest magnitude to
// [2^14, 2^15), and its inverse; 1 for rows that are zero or not finite.
__device__ __forceinline__ void kv_row_power(float top, float &up, float &down)
{
    const uint32_t e = __builtin_bit_cast(uint32_t, top) >> 23 & 0xffu; // top >= 0
    const int p = kv_clamp(127 + 14 - (int)e, -113, 100);
    const bool plain = e == 0 || e == 255;
    up = plain ? 1.0f : __builtin_bit_cast(float, (uint32_t)(127 + p) << 23);
    down = plain ? 1.0f : __builtin_bit_cast(float, (uint32_t)(127 - p) << 23);
}

} // namespace qw
