// kv_api.hip -- the C ABI of the paged int8 KV cache operators: argument
// checks on the host, then one launch (two for a split attention) on the
// caller's stream.  Nothing is allocated here, and a rejected call launches
// nothing and writes nothing.
#include <math.h>
#include <stdint.h>

#include "kv_internal.h"

namespace {

constexpr int64_t kMaxDim = 0x7fffffff;

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

struct Bytes {
    const void *p;
    uint64_t n;
};

bool meet(Bytes a, Bytes b)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return a.n && b.n && pa < pb + b.n && pb < pa + a.n;
}

// Whether any of the written ranges meets another written one or a read one.
template <size_t W, size_t R>
bool clash(const Bytes (&written)[W], const Bytes (&read)[R])
{
    for (size_t i = 0; i < W; ++i) {
        for (size_t j = i + 1; j < W; ++j)
            if (meet(written[i], written[j]))
                return true;
        for (size_t j = 0; j < R; ++j)
            if (meet(written[i], read[j]))
                return true;
    }
    return false;
}

// Rows of `width` elements of 2 bytes, `stride` apart.
struct Rows {
    const void *p;
    int64_t stride, width, count;
};

Bytes extent(Rows r)
{
    return {r.p, r.count ? (uint64_t)((r.count - 1) * r.stride + r.width) * 2u : 0u};
}

// Whether rows share an element.  Rows of one stride may interleave (the
// columns of a fused projection): they are apart where each begins behind the
// other's end within the stride.
bool rows_meet(Rows a, Rows b)
{
    if (!meet(extent(a), extent(b)))
        return false;
    if (a.stride != b.stride)
        return true;
    const int64_t bytes = a.stride * 2;
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    const int64_t shift = ((d % bytes) + bytes) % bytes; // b's column relative to a's
    return shift < a.width * 2 || shift + b.width * 2 > bytes;
}

int shift_of(int64_t block_size)
{
    switch (block_size) {
    case 16:
        return 4;
    case 32:
        return 5;
    case 64:
        return 6;
    case 128:
        return 7;
    default:
        return -1;
    }
}

bool known(int dtype) { return dtype == QW_F16 || dtype == QW_BF16; }
bool head_dim_ok(int64_t d) { return d == 64 || d == 128; }

qw_status status_of(hipError_t e) { return e == hipSuccess ? QW_SUCCESS : QW_ERROR_LAUNCH; }

struct CacheShape {
    const int8_t *k, *v;
    const float *ks, *vs;
    int64_t num_blocks, block_size, kv_heads, head_dim;
    uint64_t codes() const { return (uint64_t)num_blocks * (uint64_t)block_size * (uint64_t)kv_heads * (uint64_t)head_dim; }
    uint64_t scales() const { return (uint64_t)num_blocks * (uint64_t)kv_heads * 4u; }
};

qw_status check_cache(const CacheShape &c)
{
    if (c.num_blocks <= 0 || c.kv_heads <= 0 || !c.k || !c.v || !c.ks || !c.vs)
        return QW_ERROR_INVALID_VALUE;
    if (!head_dim_ok(c.head_dim) || shift_of(c.block_size) < 0 || c.num_blocks > kMaxDim || c.kv_heads > 65535)
        return QW_ERROR_UNSUPPORTED;
    if (off16(c.k) || off16(c.v) || off16(c.ks) || off16(c.vs))
        return QW_ERROR_MISALIGNED;
    return QW_SUCCESS;
}

int64_t smaller(int64_t a, int64_t b) { return a < b ? a : b; }

// Sizes of an attention call; kv_heads divides q_heads.  A request has as many
// queries as the call at most; 2^23 of its rows are 2^31 threads of the join.
qw_status check_attention_sizes(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t block_size,
                                int64_t table_width, int64_t requests, int64_t max_new, int64_t max_context, int64_t window)
{
    if (tokens < 0 || requests < 0 || q_heads <= 0 || kv_heads <= 0 || max_new < 0 || max_context < 0 || window < 0 ||
        table_width < 0 || q_heads % kv_heads)
        return QW_ERROR_INVALID_VALUE;
    if (!head_dim_ok(head_dim) || shift_of(block_size) < 0 || tokens > kMaxDim || requests > 65535 || q_heads > 65535 ||
        max_new > (1 << 20) || smaller(max_new, tokens) * q_heads > (1 << 23) || table_width > kMaxDim ||
        max_context > kMaxDim - 4096 || window > kMaxDim)
        return QW_ERROR_UNSUPPORTED;
    return QW_SUCCESS;
}

// What the sizes mean to the kernels: a context the table can hold, and no
// window where it hides nothing.
void settle(int64_t tokens, int64_t block_size, int64_t table_width, int64_t &max_new, int64_t &max_context, int64_t &window)
{
    max_new = smaller(max_new, tokens);
    max_context = smaller(max_context, table_width * block_size);
    if (window >= max_context + max_new)
        window = 0;
}

} // namespace

extern "C" {

QW_API qw_status qw_kv_plan(const int32_t *past, const int32_t *fresh, int64_t requests, int32_t *block_table,
                            int64_t table_width, const int32_t *free_blocks, int64_t n_free, int64_t block_size,
                            int64_t max_tokens, int32_t *cu_tokens, int32_t *context, int32_t *positions, int32_t *slots,
                            int32_t *counts, void *stream)
{
    if (requests < 0 || table_width < 0 || n_free < 0 || max_tokens < 0 || !cu_tokens || !counts ||
        (requests > 0 && (!past || !fresh || !context || (table_width > 0 && !block_table))) ||
        (n_free > 0 && !free_blocks) || (max_tokens > 0 && (!positions || !slots)))
        return QW_ERROR_INVALID_VALUE;
    const int shift = shift_of(block_size);
    if (shift < 0 || requests > QW_KV_PLAN_MAX_REQUESTS || table_width > kMaxDim || n_free > kMaxDim || max_tokens > kMaxDim)
        return QW_ERROR_UNSUPPORTED;
    if (off4(past) || off4(fresh) || off4(block_table) || off4(free_blocks) || off4(cu_tokens) || off4(context) ||
        off4(positions) || off4(slots) || off4(counts))
        return QW_ERROR_MISALIGNED;
    const uint64_t r4 = (uint64_t)requests * 4u, t4 = (uint64_t)max_tokens * 4u;
    const Bytes written[] = {{block_table, r4 * (uint64_t)table_width}, {cu_tokens, r4 + 4u}, {context, r4},
                             {positions, t4}, {slots, t4}, {counts, 8}};
    const Bytes read[] = {{past, r4}, {fresh, r4}, {free_blocks, (uint64_t)n_free * 4u}};
    if (clash(written, read))
        return QW_ERROR_INVALID_VALUE;
    const qw::KvPlanArgs a = {past, fresh, (int32_t)requests, block_table, table_width, free_blocks, (int32_t)n_free, shift,
                              (int32_t)max_tokens, cu_tokens, context, positions, slots, counts};
    return status_of(qw::launch_kv_plan(a, static_cast<hipStream_t>(stream)));
}

QW_API qw_status qw_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int dtype, int64_t tokens,
                                 int64_t q_heads, int64_t kv_heads, int64_t head_dim, const int32_t *positions, const float *cos,
                                 const float *sin, int64_t max_position, int64_t rot_dim, int interleaved, const void *q_weight,
                                 const void *k_weight, double eps, void *q_out, int64_t q_out_stride, void *k_out,
                                 int64_t k_out_stride, void *stream)
{
    if (!known(dtype) || tokens < 0 || q_heads <= 0 || kv_heads <= 0 || max_position < 0 || rot_dim < 0 || !(eps >= 0.0) ||
        !isfinite(eps) || (q_weight == nullptr) != (k_weight == nullptr))
        return QW_ERROR_INVALID_VALUE;
    if (!head_dim_ok(head_dim) || rot_dim > head_dim || rot_dim % 16 || tokens > kMaxDim || q_heads > 65535 || kv_heads > 65535 ||
        max_position > kMaxDim || tokens * (q_heads + kv_heads) > (int64_t(1) << 38) / head_dim)
        return QW_ERROR_UNSUPPORTED;
    if (tokens == 0)
        return QW_SUCCESS;
    const int64_t qw_ = q_heads * head_dim, kw = kv_heads * head_dim;
    if (!q || !k || !q_out || !k_out || !positions || (rot_dim > 0 && max_position > 0 && (!cos || !sin)) || q_stride < qw_ ||
        q_out_stride < qw_ || k_stride < kw || k_out_stride < kw)
        return QW_ERROR_INVALID_VALUE;
    const int64_t most = int64_t(1) << 31; // strides stay where tokens * stride cannot wrap
    if (q_stride % 8 || k_stride % 8 || q_out_stride % 8 || k_out_stride % 8 || q_stride > most || k_stride > most ||
        q_out_stride > most || k_out_stride > most)
        return QW_ERROR_UNSUPPORTED;
    if (off16(q) || off16(k) || off16(q_out) || off16(k_out) || off16(cos) || off16(sin) || off16(q_weight) || off16(k_weight) ||
        off4(positions))
        return QW_ERROR_MISALIGNED;
    const Rows rq = {q, q_stride, qw_, tokens}, rk = {k, k_stride, kw, tokens};
    const Rows oq = {q_out, q_out_stride, qw_, tokens}, ok = {k_out, k_out_stride, kw, tokens};
    const uint64_t table = (uint64_t)max_position * (uint64_t)(rot_dim / 2) * 4u;
    const uint64_t wb = q_weight ? (uint64_t)head_dim * 2u : 0u;
    const Bytes read[] = {{positions, (uint64_t)tokens * 4u}, {cos, table}, {sin, table}, {q_weight, wb}, {k_weight, wb}};
    const Bytes only_q[] = {extent(oq)}, only_k[] = {extent(ok)};
    const bool q_in_place = q_out == q && q_out_stride == q_stride, k_in_place = k_out == k && k_out_stride == k_stride;
    if (clash(only_q, read) || clash(only_k, read) || rows_meet(oq, ok) || rows_meet(oq, rk) || rows_meet(ok, rq) ||
        (!q_in_place && rows_meet(oq, rq)) || (!k_in_place && rows_meet(ok, rk)))
        return QW_ERROR_INVALID_VALUE;
    const qw::NormRopeArgs a = {static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k), q_stride, k_stride,
                                static_cast<uint16_t *>(q_out), static_cast<uint16_t *>(k_out), q_out_stride, k_out_stride,
                                tokens, (int32_t)q_heads, (int32_t)kv_heads, (int32_t)head_dim, positions, cos, sin, max_position,
                                (int32_t)rot_dim, interleaved != 0, static_cast<const uint16_t *>(q_weight),
                                static_cast<const uint16_t *>(k_weight), (float)eps};
    return status_of(qw::launch_qk_norm_rope(a, dtype, static_cast<hipStream_t>(stream)));
}

QW_API qw_status qw_kv_write(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, int64_t tokens,
                             int64_t kv_heads, int64_t head_dim, const int32_t *slots, int8_t *k_cache, int8_t *v_cache,
                             float *k_scales, float *v_scales, int64_t num_blocks, int64_t block_size, void *stream)
{
    if (!known(dtype) || tokens < 0)
        return QW_ERROR_INVALID_VALUE;
    const CacheShape c = {k_cache, v_cache, k_scales, v_scales, num_blocks, block_size, kv_heads, head_dim};
    const qw_status st = check_cache(c);
    if (st != QW_SUCCESS)
        return st;
    if (tokens > kMaxDim)
        return QW_ERROR_UNSUPPORTED;
    if (tokens == 0)
        return QW_SUCCESS;
    const int64_t width = kv_heads * head_dim;
    if (!k || !v || !slots || k_stride < width || v_stride < width)
        return QW_ERROR_INVALID_VALUE;
    const int64_t most = int64_t(1) << 31;
    if (k_stride % 8 || v_stride % 8 || k_stride > most || v_stride > most)
        return QW_ERROR_UNSUPPORTED;
    if (off16(k) || off16(v) || off4(slots))
        return QW_ERROR_MISALIGNED;
    const Bytes written[] = {{k_cache, c.codes()}, {v_cache, c.codes()}, {k_scales, c.scales()}, {v_scales, c.scales()}};
    const Bytes read[] = {extent({k, k_stride, width, tokens}), extent({v, v_stride, width, tokens}), {slots, (uint64_t)tokens * 4u}};
    if (clash(written, read))
        return QW_ERROR_INVALID_VALUE;
    const qw::KvCacheArgs a = {slots, tokens, (int32_t)kv_heads, (int32_t)head_dim, shift_of(block_size), num_blocks,
                               k_cache, v_cache, k_scales, v_scales, static_cast<uint16_t *>(const_cast<void *>(k)),
                               static_cast<uint16_t *>(const_cast<void *>(v)), k_stride, v_stride};
    return status_of(qw::launch_kv_write(a, dtype, static_cast<hipStream_t>(stream)));
}

QW_API qw_status qw_kv_read(const int32_t *slots, int64_t tokens, const int8_t *k_cache, const int8_t *v_cache,
                            const float *k_scales, const float *v_scales, int64_t num_blocks, int64_t block_size,
                            int64_t kv_heads, int64_t head_dim, int dtype, void *k, void *v, void *stream)
{
    if (!known(dtype) || tokens < 0)
        return QW_ERROR_INVALID_VALUE;
    const CacheShape c = {k_cache, v_cache, k_scales, v_scales, num_blocks, block_size, kv_heads, head_dim};
    const qw_status st = check_cache(c);
    if (st != QW_SUCCESS)
        return st;
    if (tokens > kMaxDim)
        return QW_ERROR_UNSUPPORTED;
    if (tokens == 0)
        return QW_SUCCESS;
    if (!k || !v || !slots)
        return QW_ERROR_INVALID_VALUE;
    if (off16(k) || off16(v) || off4(slots))
        return QW_ERROR_MISALIGNED;
    const int64_t width = kv_heads * head_dim;
    const uint64_t out = (uint64_t)tokens * (uint64_t)width * 2u;
    const Bytes written[] = {{k, out}, {v, out}};
    const Bytes read[] = {{k_cache, c.codes()}, {v_cache, c.codes()}, {k_scales, c.scales()}, {v_scales, c.scales()},
                          {slots, (uint64_t)tokens * 4u}};
    if (clash(written, read))
        return QW_ERROR_INVALID_VALUE;
    const qw::KvCacheArgs a = {slots, tokens, (int32_t)kv_heads, (int32_t)head_dim, shift_of(block_size), num_blocks,
                               const_cast<int8_t *>(k_cache), const_cast<int8_t *>(v_cache), const_cast<float *>(k_scales),
                               const_cast<float *>(v_scales), static_cast<uint16_t *>(k), static_cast<uint16_t *>(v), width, width};
    return status_of(qw::launch_kv_read(a, dtype, static_cast<hipStream_t>(stream)));
}

QW_API int64_t qw_kv_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t block_size,
                                         int64_t table_width, int64_t requests, int64_t max_new, int64_t max_context,
                                         int64_t window)
{
    if (check_attention_sizes(tokens, q_heads, kv_heads, head_dim, block_size, table_width, requests, max_new, max_context,
                              window) != QW_SUCCESS)
        return -1;
    settle(tokens, block_size, table_width, max_new, max_context, window);
    if (tokens == 0 || requests == 0 || max_new == 0)
        return 0;
    return qw::kv_attention_workspace(tokens, q_heads, kv_heads, head_dim, requests, max_new, max_context, window);
}

QW_API qw_status qw_kv_attention(const void *q, int64_t q_stride, int dtype, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                                 int64_t head_dim, const int8_t *k_cache, const int8_t *v_cache, const float *k_scales,
                                 const float *v_scales, int64_t num_blocks, int64_t block_size, const int32_t *block_table,
                                 int64_t table_width, const int32_t *context, const int32_t *cu_tokens, int64_t requests,
                                 int64_t max_new, int64_t max_context, double scale, int causal, int64_t window, void *out,
                                 void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!known(dtype) || !isfinite(scale) || workspace_bytes < 0)
        return QW_ERROR_INVALID_VALUE;
    qw_status st = check_attention_sizes(tokens, q_heads, kv_heads, head_dim, block_size, table_width, requests, max_new,
                                         max_context, window);
    if (st != QW_SUCCESS)
        return st;
    if (tokens == 0 || requests == 0 || max_new == 0)
        return QW_SUCCESS;
    const CacheShape c = {k_cache, v_cache, k_scales, v_scales, num_blocks, block_size, kv_heads, head_dim};
    st = check_cache(c);
    if (st != QW_SUCCESS)
        return st;
    const int64_t width = q_heads * head_dim;
    if (!q || !out || !context || !cu_tokens || (table_width > 0 && !block_table) || q_stride < width)
        return QW_ERROR_INVALID_VALUE;
    if (q_stride % 8 || q_stride > (int64_t(1) << 31))
        return QW_ERROR_UNSUPPORTED;
    if (off16(q) || off16(out) || off16(workspace) || off4(block_table) || off4(context) || off4(cu_tokens))
        return QW_ERROR_MISALIGNED;
    settle(tokens, block_size, table_width, max_new, max_context, window);
    const int64_t need = qw::kv_attention_workspace(tokens, q_heads, kv_heads, head_dim, requests, max_new, max_context, window);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return QW_ERROR_INVALID_VALUE;
    const Bytes written[] = {{out, (uint64_t)tokens * (uint64_t)width * 2u}, {workspace, (uint64_t)need}};
    const Bytes read[] = {extent({q, q_stride, width, tokens}), {k_cache, c.codes()}, {v_cache, c.codes()}, {k_scales, c.scales()},
                          {v_scales, c.scales()}, {block_table, (uint64_t)requests * (uint64_t)table_width * 4u},
                          {context, (uint64_t)requests * 4u}, {cu_tokens, (uint64_t)(requests + 1) * 4u}};
    if (clash(written, read))
        return QW_ERROR_INVALID_VALUE;
    const qw::KvAttnArgs a = {static_cast<const uint16_t *>(q), q_stride, static_cast<uint16_t *>(out), (int32_t)tokens,
                              (int32_t)q_heads, (int32_t)kv_heads, (int32_t)(q_heads / kv_heads), (int32_t)head_dim, k_cache, v_cache,
                              k_scales, v_scales, num_blocks, shift_of(block_size), block_table, (int32_t)table_width, context,
                              cu_tokens, (int32_t)requests, (int32_t)max_new, (int32_t)max_context,
                              (float)(scale * 1.4426950408889634), (causal & ~QW_KV_ZERO_REST) != 0, (int32_t)window, static_cast<float *>(workspace),
                              (causal & QW_KV_ZERO_REST) != 0};
    return status_of(qw::launch_kv_attention(a, dtype, static_cast<hipStream_t>(stream)));
}

} // extern "C"
