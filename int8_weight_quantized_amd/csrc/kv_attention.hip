// kv_attention.hip -- attention over the paged int8 KV cache.
//
// For the query row i of a request's n new tokens (of `context` cached ones,
// the new ones among them) at position p = context - n + i, and the keys j
// it may see (j < context; j <= p if causal; j > p - window if windowed):
//
//   s_j = scale * Sk(j) * sum_d q_d Kq[j][d]
//   o_d = sum_j e^{s_j} Sv(j) Vq[j][d] / sum_j e^{s_j}        (no key: 0)
//
// with Sk, Sv the scales of key j's block.  int8 codes are exact in fp16, so
// both products run on the fp16 matrix cores: Q Kq^T with q as given (bf16
// rows are first multiplied by a power of two that brings their largest
// element to [2^14, 2^15), which makes the cast to fp16 exact for elements
// down to 2^-29 of it), and P Vq with P rounded to fp16.
//
// The value scale is folded into the softmax's exponent:
//   t_j = log2(e) s_j + log2 Sv(j),  P_j = 2^{t_j - M},  M >= max t_j - 8
//   o = sum P_j Vq[j] / sum (P_j / Sv(j))
// so one running reference M serves both sums, P stays within 2^8 whatever
// the scales of the blocks, and the denominator needs one multiplication per
// 16 keys.  M moves only when a row's maximum has grown by 2^8 or more; the
// accumulators are rescaled then.  M, the denominators and the accumulators
// are fp32.
//
// Query rows that share a key head (the heads of its group, for each new
// token) form the columns of one matrix product, so the cache is read once
// for all of them.
#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64; // keys a wave takes at once
constexpr float kLazy = 8.0f;

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// What a block of query rows of one request attends to.
struct Span {
    int t0, past; // first token; cached tokens before it (negative where there are more queries than cached tokens)
    int ctx;      // cached tokens
    int rows;     // query rows of a key head: those of at most max_new tokens
    int lo, hi;   // keys any of the rows [row0, row0 + count) sees; lo is a multiple of kTile
};

__device__ __forceinline__ Span span_of(const KvAttnArgs &a, int r, int row0, int count)
{
    Span s;
    s.t0 = clampi(a.cu_tokens[r], 0, a.tokens);
    const int n = clampi(a.cu_tokens[r + 1], s.t0, a.tokens) - s.t0;
    s.ctx = clampi(a.context[r], 0, a.max_context);
    s.past = s.ctx - n;
    s.rows = (n < a.max_new ? n : a.max_new) * a.group;
    s.lo = s.hi = 0;
    if (row0 < s.rows) {
        const int end = row0 + count < s.rows ? row0 + count : s.rows;
        const int first = row0 / a.group, last = (end - 1) / a.group;
        s.hi = a.causal ? clampi(s.past + last + 1, 0, s.ctx) : s.ctx;
        s.lo = a.window ? clampi(s.past + first - a.window + 1, 0, s.hi) & ~(kTile - 1) : 0;
    }
    return s;
}

// 8 activations -> fp16 (bf16 after multiplication by `up`, a power of two).
template <int DT>
__device__ __forceinline__ half8_t to_half8(u32x4_t v, float up)
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
__device__ __forceinline__ void row_power(float top, float &up, float &down)
{
    const uint32_t e = __builtin_bit_cast(uint32_t, top) >> 23 & 0xffu; // top >= 0
    const int p = clampi(127 + 14 - (int)e, -113, 100);
    const bool plain = e == 0 || e == 255;
    up = plain ? 1.0f : __builtin_bit_cast(float, (uint32_t)(127 + p) << 23);
    down = plain ? 1.0f : __builtin_bit_cast(float, (uint32_t)(127 - p) << 23);
}

// ---------------------------------------------------------------------------
// Split kernel: one workgroup for a chunk of the context, a key head and a
// block of 16 RT query rows; its four waves take the chunk's 64-key tiles in
// turn and are joined through LDS at the end.
//
// S^T = Kq Q^T and O^T = Vq^T P^T on v_mfma_f32_16x16x32_f16.  A lane holds
// column (query row) lane & 15 of S^T; which keys its registers hold depends
// only on which cache rows fed the first product, and they are chosen so
// that lane group g = lane / 16 holds keys 16 g .. 16 g + 15 of the tile:
// exactly the operand layout of the second product, whose other operand is
// then one contiguous 16-byte load a lane from the transposed values.
// Nothing passes through LDS or between lanes but the row maximum.
//
// Bound by HBM: 2 * D + 8 / B bytes a key and head, each read once, straight
// into registers; a tile is D / 4 16-byte loads in flight a lane.
// ---------------------------------------------------------------------------
template <int D, int RT, int DT, bool WIDE /* a tile lies in one block */>
__global__ __launch_bounds__(kThreads, RT == 1 ? 3 : 2) void kv_split_kernel(KvAttnArgs a, int chunk, int chunks)
{
    constexpr int CH = D / 64;  // 64-channel pieces of a key row
    constexpr int DTILES = D / 16;
    constexpr int PITCH = D + 4;
    __shared__ __attribute__((aligned(16))) float lds_o[4 * 16 * PITCH];
    __shared__ float lds_m[4][16 * RT], lds_l[4][16 * RT];

    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int kvh = blockIdx.y % a.kv_heads, rb = blockIdx.y / a.kv_heads, r = blockIdx.z;
    const int row0 = rb * 16 * RT;
    const Span s = span_of(a, r, row0, 16 * RT);
    if (row0 >= s.rows)
        return;
    const int begin = s.lo + (int)blockIdx.x * chunk;
    if (begin >= s.hi && blockIdx.x > 0)
        return;
    const int end = s.hi - begin < chunk ? s.hi : begin + chunk;

    // query rows, as the first product's second operand
    half8_t q[RT][CH][2];
    float mult[RT]; // scores -> exponents of 2, without the key scale
    int lim_lo[RT], lim_hi[RT];
    const int past = s.past;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = row0 + t * 16 + col;
        const bool in = row < s.rows;
        const int i = in ? row / a.group : 0, head = kvh * a.group + (in ? row - i * a.group : 0);
        const uint16_t *src = a.q + (int64_t)(s.t0 + i) * a.q_stride + (int64_t)head * D + g * 16;
        u32x4_t raw[CH][2];
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                raw[c][h] = in ? *reinterpret_cast<const u32x4_t *>(src + c * 64 + h * 8) : (u32x4_t){0, 0, 0, 0};
                if (DT == QW_BF16) {
                    float f[8];
                    unpack8<DT>(raw[c][h], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        top = fmaxf(top, fabsf(f[e]));
                }
            }
        float up = 1.0f, down = 1.0f;
        if (DT == QW_BF16)
            row_power(max_xor32(max_xor16(top)), up, down);
        mult[t] = a.scale_log2 * down;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[t][c][h] = to_half8<DT>(raw[c][h], up);
        lim_hi[t] = in ? (a.causal ? past + i + 1 : s.ctx) : 0;
        lim_lo[t] = a.window ? past + i - a.window + 1 : 0;
    }
    // keys that every row of the block sees
    const int last_row = row0 + 16 * RT < s.rows ? row0 + 16 * RT - 1 : s.rows - 1;
    const int all_hi = a.causal ? past + row0 / a.group + 1 : s.ctx;
    const int all_lo = a.window ? past + last_row / a.group - a.window + 1 : 0;

    float4_t o[RT][DTILES];
    float m[RT], l[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
            o[t][d] = (float4_t){0, 0, 0, 0};
    }

    const int32_t *table = a.block_table + (int64_t)r * a.table_width;
    const int block = 1 << a.block_shift;
    const int64_t head_bytes = (int64_t)block * D;
    // Cache block that holds key j (0 where the table holds none: it is read
    // in its place and masked).
    auto block_of = [&](int j, bool &ok) {
        int32_t id = j < s.hi ? table[j >> a.block_shift] : -1;
        ok = id >= 0 && id < a.num_blocks;
        return (int64_t)(ok ? id : 0) * a.kv_heads + kvh;
    };

    u32x4_t kraw[4][CH], vraw[DTILES];
    float ks, vs;
    bool ok;
    auto load = [&](int base) {
        // key rows: row c of 16-key product i is key 16 (c / 4) + 4 i + c % 4
        int64_t kb, vb;
        if (WIDE) {
            kb = vb = block_of(base, ok);
        } else {
            bool unused;
            kb = block_of(base + (col >> 2) * 16, unused);
            vb = block_of(base + g * 16, ok);
        }
        const int8_t *kp = a.k_cache + kb * head_bytes +
                           (int64_t)(((base + (col >> 2) * 16) & (block - 1)) + (col & 3)) * D + g * 16;
        const int8_t *vp = a.v_cache + vb * head_bytes + (int64_t)col * block + ((base + g * 16) & (block - 1));
        ks = a.k_scales[vb];
        vs = a.v_scales[vb];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                kraw[i][c] = *reinterpret_cast<const u32x4_t *>(kp + i * 4 * D + c * 64);
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
            vraw[d] = *reinterpret_cast<const u32x4_t *>(vp + (int64_t)d * 16 * block);
    };

    for (int base = begin + wave * kTile; base < end; base += 4 * kTile) {
        load(base);
        float4_t sc[RT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
                sc[t][i] = (float4_t){0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const half8_t k0 = i8x8_to_half8(kraw[i][c].x, kraw[i][c].y);
                const half8_t k1 = i8x8_to_half8(kraw[i][c].z, kraw[i][c].w);
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    sc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q[t][c][0], sc[t][i], 0, 0, 0);
                    sc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q[t][c][1], sc[t][i], 0, 0, 0);
                }
            }
        }
        const bool whole = base >= all_lo && base + kTile <= all_hi && __all(ok);
        const float vsc = fmaxf(vs, kKvScaleFloor);
        const float lv = ok ? __log2f(vsc) : 0.0f;
        const float inv = ok ? 1.0f / vsc : 0.0f;
        half8_t p[RT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const float c = ok ? mult[t] * ks : 0.0f;
            float x[16];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[4 * i + j] = fmaf(sc[t][i][j], c, lv);
            if (!whole) {
                const int at = base + g * 16;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = ok && at + e >= lim_lo[t] && at + e < lim_hi[t] ? x[e] : -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
                top = fmaxf(top, x[e]);
            top = max_xor32(max_xor16(top));
            if (__any(top > m[t] + kLazy)) {
                const float next = fmaxf(m[t], top);
                const float alpha = next == m[t] ? 1.0f : __builtin_amdgcn_exp2f(m[t] - next);
                m[t] = next;
                l[t] *= alpha;
#pragma unroll
                for (int d = 0; d < DTILES; ++d)
                    o[t][d] *= alpha;
            }
            const float ref = m[t] == -INFINITY ? 0.0f : m[t];
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float w = __builtin_amdgcn_exp2f(x[e] - ref);
                sum += w;
                p[t][e >> 3][e & 7] = (_Float16)w; // to nearest: 2^-12 of a weight
            }
            l[t] = fmaf(sum, inv, l[t]);
        }
#pragma unroll
        for (int d = 0; d < DTILES; ++d) {
            const half8_t v0 = i8x8_to_half8(vraw[d].x, vraw[d].y);
            const half8_t v1 = i8x8_to_half8(vraw[d].z, vraw[d].w);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[t][0], o[t][d], 0, 0, 0);
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[t][1], o[t][d], 0, 0, 0);
            }
        }
    }

    // join the waves, one 16-row tile at a time
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] = add_xor32(add_xor16(l[t]));
        if (g == 0) {
            lds_m[wave][t * 16 + col] = m[t];
            lds_l[wave][t * 16 + col] = l[t];
        }
    }
    __syncthreads();
    const int valid = (s.hi - s.lo + chunk - 1) / chunk; // chunks of this row block
    const bool final = valid <= 1;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        float ref = lds_m[0][t * 16 + col];
#pragma unroll
        for (int w = 1; w < 4; ++w)
            ref = fmaxf(ref, lds_m[w][t * 16 + col]);
        const float f = m[t] == ref ? 1.0f : __builtin_amdgcn_exp2f(m[t] - ref);
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
            *reinterpret_cast<float4_t *>(lds_o + (wave * 16 + col) * PITCH + d * 16 + g * 4) = o[t][d] * f;
        __syncthreads();
        // 16 threads a row, D / 16 channels each
        const int row = (int)threadIdx.x >> 4, d0 = ((int)threadIdx.x & 15) * (D / 16);
        float rm = lds_m[0][t * 16 + row], rl = 0.0f;
#pragma unroll
        for (int w = 1; w < 4; ++w)
            rm = fmaxf(rm, lds_m[w][t * 16 + row]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float mw = lds_m[w][t * 16 + row];
            rl += lds_l[w][t * 16 + row] * (mw == rm ? 1.0f : __builtin_amdgcn_exp2f(mw - rm));
        }
        float acc[D / 16];
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
            acc[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                acc[e] += lds_o[(w * 16 + row) * PITCH + d0 + e];
        }
        const int gr = row0 + t * 16 + row;
        if (gr < s.rows) {
            if (final) {
                const int i = gr / a.group, head = kvh * a.group + gr - i * a.group;
                const float n = rl == 0.0f ? 0.0f : 1.0f / rl;
                uint32_t *out = reinterpret_cast<uint32_t *>(a.out + ((int64_t)(s.t0 + i) * a.q_heads + head) * D + d0);
#pragma unroll
                for (int e = 0; e < D / 16; e += 2)
                    out[e / 2] = Act<DT>::pack(acc[e] * n, acc[e + 1] * n);
            } else {
                const int64_t part =
                    (((int64_t)r * gridDim.y + blockIdx.y) * chunks + blockIdx.x) * (16 * RT) + t * 16 + row;
                float *w = a.workspace + part * (D + 4); // D channels, then M and the denominator
#pragma unroll
                for (int e = 0; e < D / 16; e += 4)
                    *reinterpret_cast<float4_t *>(w + d0 + e) = (float4_t){acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
                if (d0 == 0) {
                    w[D] = rm;
                    w[D + 1] = rl;
                }
            }
        }
        if (t + 1 < RT)
            __syncthreads();
    }
}

// Joins the chunks of a row: one wave a row, its lanes over the channels.
template <int D, int RT, int DT>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(KvAttnArgs a, int chunk, int chunks, int row_blocks)
{
    constexpr int E = D / 64;
    const int lane = __lane_id(), wave = (int)threadIdx.x >> 6;
    const int row = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + wave);
    const int kvh = blockIdx.y, r = blockIdx.z;
    const int rb = row / (16 * RT);
    const Span s = span_of(a, r, rb * 16 * RT, 16 * RT);
    if (row >= s.rows)
        return;
    int valid = (s.hi - s.lo + chunk - 1) / chunk;
    if (valid <= 1)
        return; // written by its only workgroup
    valid = valid < chunks ? valid : chunks;
    const int64_t unit = (int64_t)r * row_blocks * a.kv_heads + rb * a.kv_heads + kvh;
    const float *w = a.workspace + (unit * chunks * (16 * RT) + (row - rb * 16 * RT)) * (D + 4);
    const int64_t step = (int64_t)(16 * RT) * (D + 4);
    float ref = -INFINITY;
    for (int c = lane; c < valid; c += 64)
        ref = fmaxf(ref, w[c * step + D]);
    ref = wave_max_f32(ref);
    float l = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.0f;
    for (int c = 0; c < valid; ++c) {
        const float *p = w + c * step;
        const float f = p[D] == ref ? 1.0f : __builtin_amdgcn_exp2f(p[D] - ref);
        l = fmaf(p[D + 1], f, l);
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = fmaf(p[lane * E + e], f, acc[e]);
    }
    const float n = l == 0.0f ? 0.0f : 1.0f / l;
    const int i = row / a.group, head = kvh * a.group + row - i * a.group;
    uint16_t *out = a.out + ((int64_t)(s.t0 + i) * a.q_heads + head) * D + lane * E;
    if (E == 2)
        *reinterpret_cast<uint32_t *>(out) = Act<DT>::pack(acc[0] * n, acc[E - 1] * n);
    else
        *out = (uint16_t)Act<DT>::pack(acc[0] * n, 0.0f);
}

struct SplitShape {
    int rt, row_blocks, chunk, chunks;
};

SplitShape split_shape(int64_t requests, int64_t kv_heads, int64_t group, int64_t max_new, int64_t max_context,
                       int64_t window)
{
    SplitShape p;
    const int64_t rows = max_new * group;
    p.rt = rows <= 16 ? 1 : 2;
    p.row_blocks = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    int64_t span = max_context;
    if (window && window + max_new + kTile < span)
        span = window + max_new + kTile;
    const int64_t units = requests * kv_heads * p.row_blocks;
    const int64_t want = (1536 + units - 1) / units;
    const int64_t step = 4 * kTile;
    int64_t chunk = ((span + want - 1) / want + step - 1) / step * step;
    if (span <= 512)
        chunk = 512;
    p.chunk = (int)(chunk < step ? step : chunk);
    p.chunks = (int)((span + p.chunk - 1) / p.chunk);
    if (p.chunks < 1)
        p.chunks = 1;
    return p;
}

template <int D, int RT, int DT>
hipError_t launch_split(const KvAttnArgs &a, const SplitShape &p, hipStream_t stream)
{
    const dim3 grid((unsigned)p.chunks, (unsigned)(p.row_blocks * a.kv_heads), (unsigned)a.requests);
    if (a.block_shift >= 6)
        kv_split_kernel<D, RT, DT, true><<<grid, dim3(kThreads), 0, stream>>>(a, p.chunk, p.chunks);
    else
        kv_split_kernel<D, RT, DT, false><<<grid, dim3(kThreads), 0, stream>>>(a, p.chunk, p.chunks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.chunks == 1)
        return e;
    const int rows = a.max_new * a.group;
    kv_join_kernel<D, RT, DT><<<dim3((unsigned)((rows + 3) / 4), (unsigned)a.kv_heads, (unsigned)a.requests),
                                dim3(kThreads), 0, stream>>>(a, p.chunk, p.chunks, p.row_blocks);
    return hipGetLastError();
}

template <int D, int DT>
hipError_t launch_dim(const KvAttnArgs &a, hipStream_t stream)
{
    const SplitShape p = split_shape(a.requests, a.kv_heads, a.group, a.max_new, a.max_context, a.window);
    return p.rt == 1 ? launch_split<D, 1, DT>(a, p, stream) : launch_split<D, 2, DT>(a, p, stream);
}

} // namespace

int64_t kv_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                               int64_t requests, int64_t max_new, int64_t max_context, int64_t window)
{
    const SplitShape p = split_shape(requests, kv_heads, q_heads / kv_heads, max_new, max_context, window);
    if (p.chunks == 1)
        return 0;
    return requests * kv_heads * p.row_blocks * p.chunks * (16 * p.rt) * (head_dim + 4) * (int64_t)sizeof(float);
}

hipError_t launch_kv_attention(const KvAttnArgs &a, int dtype, hipStream_t stream)
{
    if (a.head_dim == 64)
        return dtype == QW_F16 ? launch_dim<64, QW_F16>(a, stream) : launch_dim<64, QW_BF16>(a, stream);
    if (a.head_dim == 128)
        return dtype == QW_F16 ? launch_dim<128, QW_F16>(a, stream) : launch_dim<128, QW_BF16>(a, stream);
    return hipErrorInvalidValue;
}

} // namespace qw
