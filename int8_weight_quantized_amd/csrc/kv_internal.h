// kv_internal.h -- parameters and host-side launchers of the paged int8 KV
// cache operators, shared between their translation units.  Arguments
// reaching the launchers have been validated by kv_api.hip.
//
// One layer's cache: k_cache [blocks][kv_heads][block_size][head_dim] and
// v_cache [blocks][kv_heads][head_dim][block_size] int8 codes, k_scales and
// v_scales [blocks][kv_heads] fp32; a value is code * scale.  The values of
// a block are stored transposed so that a lane of the attention kernels
// reads consecutive tokens of one channel, the layout the second matrix
// product's operand has, with one 16-byte load.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qw.h"

namespace qw {

// A block whose scale would lie below this holds zero codes and scale 0:
// the attention kernels divide a probability by the value scale, and with
// this floor that stays inside binary32.
constexpr float kKvScaleFloor = 7.88860905221011805411728565282786e-31f; // 2^-100

struct KvPlanArgs {
    const int32_t *past, *fresh;
    int32_t requests;
    int32_t *block_table;
    int64_t table_width;
    const int32_t *free_blocks;
    int32_t n_free;
    int32_t block_shift;
    int32_t max_tokens;
    int32_t *cu_tokens, *context, *positions, *slots, *counts;
};
hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t stream);

struct NormRopeArgs {
    const uint16_t *q, *k;
    int64_t q_stride, k_stride; // elements between tokens
    uint16_t *q_out, *k_out;
    int64_t q_out_stride, k_out_stride;
    int64_t tokens;
    int32_t q_heads, kv_heads, head_dim;
    const int32_t *positions;
    const float *cos, *sin;
    int64_t max_position;
    int32_t rot_dim;
    bool interleaved;
    const uint16_t *q_weight, *k_weight; // both null: no norm
    float eps;
};
hipError_t launch_qk_norm_rope(const NormRopeArgs &a, int dtype, hipStream_t stream);

struct KvCacheArgs {
    const int32_t *slots;
    int64_t tokens;
    int32_t kv_heads, head_dim, block_shift;
    int64_t num_blocks;
    int8_t *k_cache, *v_cache;
    float *k_scales, *v_scales;
    uint16_t *k, *v; // read by the write, written by the read
    int64_t k_stride, v_stride;
};
hipError_t launch_kv_write(const KvCacheArgs &a, int dtype, hipStream_t stream);
hipError_t launch_kv_read(const KvCacheArgs &a, int dtype, hipStream_t stream);

struct KvAttnArgs {
    const uint16_t *q;
    int64_t q_stride;
    uint16_t *out; // [tokens][q_heads][head_dim]
    int32_t tokens, q_heads, kv_heads, group, head_dim;
    const int8_t *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    int64_t num_blocks;
    int32_t block_shift;
    const int32_t *block_table;
    int32_t table_width; // entries of a row
    const int32_t *context, *cu_tokens;
    int32_t requests, max_new, max_context;
    float scale_log2; // softmax scale * log2(e)
    int32_t causal, window;
    float *workspace;
    bool zero_rest = false;                         // rows of `out` that no request computes become zero
    int32_t least_rows = 0, most_rows = 0x7fffffff; // rows a key head of the requests that a launch takes
};
int device_cu_count(); // qw_api.hip

// Workspace bytes of the shape's split along the context (0: none).
int64_t kv_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                               int64_t requests, int64_t max_new, int64_t max_context, int64_t window);
hipError_t launch_kv_attention(const KvAttnArgs &a, int dtype, hipStream_t stream);
// The kernel for many query rows (kv_prompt.hip): 128 channels, else any sizes.
hipError_t launch_kv_prompt(const KvAttnArgs &a, int dtype, hipStream_t stream);

} // namespace qw
