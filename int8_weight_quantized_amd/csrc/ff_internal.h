// ff_internal.h -- host-side launchers of the norm, the router and the sum
// over experts.  Arguments have been checked by ff_api.hip.
#pragma once

#include "qw_internal.h"

namespace qw {

struct AddNormArgs {
    const uint16_t *x, *residual, *weight; // residual null: nothing is added
    uint16_t *h;                           // null without a residual
    uint16_t *y;                           // or, null:
    int8_t *q;
    uint16_t *scales;
    int64_t x_stride, residual_stride, h_stride; // elements between rows
    int64_t tokens, k;
    float eps;
};
hipError_t launch_add_rms_norm(const AddNormArgs &a, int dtype, hipStream_t stream);

struct RouteArgs {
    const void *logits; // [tokens][experts]
    const float *bias;  // [experts], or null
    int64_t tokens;
    int experts, top_k, sigmoid, groups, top_groups, renormalize;
    double scale;
    int32_t *ids;      // [tokens][top_k]
    float *weights;    // [tokens][top_k]
    int32_t *offsets;  // [experts + 1]
    int32_t *rows;     // [tokens * top_k]
    int32_t *places;   // [tokens][top_k]
    int32_t *counts;   // workspace: [blocks][counts_stride]
    int counts_stride; // experts, up to a multiple of 4
    int tokens_a_block; // route_tokens_a_block()
    int blocks;         // that have tokens
};
// Tokens of one workgroup's share.
int64_t route_tokens_a_block(int64_t tokens);
hipError_t launch_route_experts(const RouteArgs &a, int dtype, hipStream_t stream);

struct CombineArgs {
    const void *y;           // fp16 or, `f32`, fp32 [entries][n]
    const int32_t *places;   // [tokens][top_k]
    const float *weights;    // [tokens][top_k]
    const uint16_t *residual; // fp16 [tokens][n], or null
    uint16_t *out;           // fp16 [tokens][n]
    int64_t tokens, entries, n;
    int top_k;
    bool f32;
};
hipError_t launch_experts_combine(const CombineArgs &a, hipStream_t stream);

} // namespace qw
