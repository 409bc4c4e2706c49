// kv_prompt.hip -- attention over the paged int8 KV cache for many query rows
// (prompts and chunks of them).  The formulas, the fold of the value scales
// into the exponent and the reference M are those of kv_attention.hip.
//
// A workgroup of eight waves takes 256 query rows that share a key head (the
// heads of its group, for consecutive tokens): 32 rows a wave, the columns of
// S^T = Kq Q^T and O^T = Vq^T P^T on v_mfma_f32_32x32x16_f16.  A lane holds
// half of the keys of one row, so a row's maximum is one exchange between
// lane halves, and P leaves the softmax in the registers in which the second
// product wants it: the order of the key rows in the first product is chosen
// so that registers 8 j .. 8 j + 7 of lane half h hold keys 16 j + 8 h + 0..7.
//
// Tiles of 64 keys are cast to fp16 once, on their way into LDS, by all eight
// waves (16 bytes of codes a thread and operand), and are read from there by
// each wave in whole fragments of the matrix instruction: fragment f is 1 KiB,
// 16 bytes a lane, lane l's piece in slot l ^ x with x the fragment's position
// along the contiguous direction of the cache, so that both the reads (a
// permutation of one KiB) and the writes (eight lanes hold consecutive pieces
// of one row, that is eight fragments) touch all banks evenly.  Two buffers;
// one barrier a tile.
//
// Bound by the matrix cores together with the softmax's VALU work: per tile
// and wave 2 * D / 4 matrix instructions of 32 cycles, and for each of 32
// scores a lane one FMA, half a maximum, one exponential at a quarter of the
// rate, one addition and half a conversion.
#include "kv_attention_device.h"

namespace qw {

namespace {

constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves; // query rows of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 64;
constexpr float kLazy = 8.0f;
constexpr float kNothing = -3e38f; // the threshold of a row that has seen no key

template <int D>
union PromptLds {
    struct {
        half8_t k[2][kTile * D / 8]; // [32-key half][16-channel step][slot]
        half8_t v[2][kTile * D / 8]; // [32-channel tile][16-key step][slot]
        float4_t scale[2][4];        // per 16 keys: key scale * log2(e) * softmax scale, log2 of the value scale, its inverse
    };
    uint16_t out[kRows][D + 8];
};

template <int D, int DT>
__global__ __launch_bounds__(kThreads, 2) void kv_prompt_kernel(KvAttnArgs a, int row_blocks)
{
    constexpr int STEPS = D / 16; // of the first product
    constexpr int DTILES = D / 32;
    __shared__ __attribute__((aligned(16))) PromptLds<D> lds;

    const int tid = threadIdx.x, lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;
    // row blocks from the last to the first: under a causal mask the longest first
    const int per_block = a.requests * a.kv_heads;
    const int rb = row_blocks - 1 - (int)blockIdx.x / per_block;
    const int unit = (int)blockIdx.x % per_block;
    const int r = unit / a.kv_heads, kvh = unit - r * a.kv_heads;
    const KvRequest s = kv_request(a, r);
    const int row0 = rb * kRows;
    if (row0 >= s.rows)
        return;
    const int last_row = row0 + kRows < s.rows ? row0 + kRows - 1 : s.rows - 1;
    const int first_i = row0 / a.group, last_i = last_row / a.group;
    // keys that some row of the block sees, and keys that every one does
    const int end = a.causal ? kv_clamp(s.past + last_i + 1, 0, s.ctx) : s.ctx;
    const int begin = a.window ? kv_clamp(s.past + first_i - a.window + 1, 0, end) & ~(kTile - 1) : 0;
    const int all_hi = a.causal ? s.past + first_i + 1 : s.ctx;
    const int all_lo = a.window ? s.past + last_i - a.window + 1 : 0;

    // ---- staging: what this thread brings into LDS -------------------------
    const int block = 1 << a.block_shift;
    const int64_t head_bytes = (int64_t)block * D;
    const int32_t *table = a.block_table + (int64_t)r * a.table_width;
    constexpr int KP = kTile * D / 16; // 16-byte pieces of an operand's tile
    constexpr bool kBoth = KP == kThreads; // a piece of each a thread; otherwise half the threads bring keys, half values
    const bool brings_k = kBoth || tid < KP, brings_v = kBoth || tid >= KP;
    const int kp = kBoth ? tid : (tid & (KP - 1)); // which piece
    const int kt = kp / (D / 16), kc = kp % (D / 16); // key of the tile, 16-channel step
    const int vd = kp >> 2, vk = kp & 3;            // channel, 16-key step
    const int kgroup = kt >> 4;
    // slots: row m of the first product's tile holds key u of 32
    const int u = kt & 31;
    const int m = (u & 3) + 16 * (u >> 4) + 8 * ((u >> 2) & 1) + 4 * ((u >> 3) & 1);
    const int kslot = ((kt >> 5) * STEPS + kc) * 64, vslot = ((vd >> 5) * 4 + vk) * 64;
    const int k0 = kslot + (m ^ (kc & 7)), k1 = kslot + ((m + 32) ^ (kc & 7));
    const int v0 = vslot + ((vd & 31) ^ (vk << 1)), v1 = vslot + (((vd & 31) + 32) ^ (vk << 1));

    auto look = [&](int j) { return j < end ? table[j >> a.block_shift] : -1; };
    auto known = [&](int32_t id) { return id >= 0 && id < a.num_blocks; };
    auto row_of = [&](int32_t id) { return (int64_t)(known(id) ? id : 0) * a.kv_heads + kvh; };
    u32x4_t kraw = {0, 0, 0, 0}, vraw = {0, 0, 0, 0};
    float ks = 0.0f, vs = 0.0f;
    bool ok = false;
    int32_t kid = -1, vid = -1, sid = -1; // blocks of this thread's pieces and of 16-key group tid % 4
    auto look_all = [&](int base) {
        kid = brings_k ? look(base + kgroup * 16) : -1;
        vid = brings_v ? look(base + vk * 16) : -1;
        sid = look(base + (tid & 3) * 16);
    };
    auto load = [&](int base) {
        if (brings_k)
            kraw = *reinterpret_cast<const u32x4_t *>(a.k_cache + row_of(kid) * head_bytes +
                                                      (uint32_t)(((base + kt) & (block - 1)) * D + kc * 16));
        if (brings_v)
            vraw = *reinterpret_cast<const u32x4_t *>(a.v_cache + row_of(vid) * head_bytes +
                                                      (uint32_t)(vd * block + ((base + vk * 16) & (block - 1))));
        ks = a.k_scales[row_of(sid)];
        vs = a.v_scales[row_of(sid)];
        ok = known(sid);
    };
    auto store = [&](int buf) {
        if (brings_k) {
            lds.k[buf][k0] = i8x8_to_half8(kraw.x, kraw.y);
            lds.k[buf][k1] = i8x8_to_half8(kraw.z, kraw.w);
        }
        if (brings_v) {
            lds.v[buf][v0] = i8x8_to_half8(vraw.x, vraw.y);
            lds.v[buf][v1] = i8x8_to_half8(vraw.z, vraw.w);
        }
        if (tid < 4) {
            const float sc = fmaxf(vs, kKvScaleFloor);
            // (a group without a block: scores of -inf, whatever its codes)
            lds.scale[buf][tid] = ok ? (float4_t){ks * a.scale_log2, __log2f(sc), 1.0f / sc, 0.0f}
                                     : (float4_t){0.0f, -INFINITY, 0.0f, 0.0f};
        }
    };

    look_all(begin);
    if (begin < end)
        load(begin);

    // ---- this wave's query rows --------------------------------------------
    const int row = row0 + wave * 32 + col;
    const bool in = row < s.rows;
    const int qi = in ? row / a.group : 0, head = kvh * a.group + (in ? row - qi * a.group : 0);
    half8_t q[STEPS];
    float down = 1.0f;
    {
        const uint16_t *src = a.q + (int64_t)(s.t0 + qi) * a.q_stride + (int64_t)head * D + h * 8;
        u32x4_t raw[STEPS];
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < STEPS; ++c) {
            raw[c] = in ? *reinterpret_cast<const u32x4_t *>(src + c * 16) : (u32x4_t){0, 0, 0, 0};
            if (DT == QW_BF16) {
                float f[8];
                unpack8<DT>(raw[c], f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, fabsf(f[e]));
            }
        }
        float up = 1.0f;
        if (DT == QW_BF16)
            kv_row_power(max_xor32(top), up, down);
#pragma unroll
        for (int c = 0; c < STEPS; ++c)
            q[c] = kv_half8<DT>(raw[c], up);
    }
    const int lim_hi = in ? (a.causal ? s.past + qi + 1 : s.ctx) : 0;
    const int lim_lo = a.window ? s.past + qi - a.window + 1 : 0;

    float16_t o[DTILES];
#pragma unroll
    for (int d = 0; d < DTILES; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[d][i] = 0.0f;
    // A row's reference moves when a score exceeds it by the threshold: kLazy,
    // or anything while the row has seen no key.
    float ref = 0.0f, above = kNothing, l = 0.0f;

    look_all(begin + kTile);
    if (begin < end)
        store(0);
    __syncthreads();

    int buf = 0;
    for (int base = begin; base < end; base += kTile, buf ^= 1) {
        const bool more = base + kTile < end;
        if (more) {
            load(base + kTile);
            look_all(base + 2 * kTile);
        }

        float16_t sc[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sc[t][i] = 0.0f;
#pragma unroll
            for (int c = 0; c < STEPS; ++c)
                sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lds.k[buf][(t * STEPS + c) * 64 + (lane ^ (c & 7))], q[c], sc[t],
                                                               0, 0, 0);
        }

        // exponents relative to the reference; 8 scores a lane share a scale
        float4_t g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            g[j] = lds.scale[buf][j];
        const bool whole = base >= all_lo && base + kTile <= all_hi;
        float x[32];
        auto exponents = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float c = g[j].x * down, b = g[j].y - ref;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[8 * j + e] = fmaf(sc[j >> 1][(j & 1) * 8 + e], c, b);
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int at = base + j * 16 + h * 8 + e;
                        x[8 * j + e] = at >= lim_lo && at < lim_hi ? x[8 * j + e] : -INFINITY;
                    }
            }
        };
        exponents();
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 32; ++e)
            top = fmaxf(top, x[e]);
        if (__any(top > above)) {
            top = max_xor32(top);
            const bool first = above == kNothing, seen = top > kNothing;
            const float up = first ? (seen ? top : 0.0f) : fmaxf(top, 0.0f); // the new reference lies so far above the old
            const float alpha = first ? 1.0f : __builtin_amdgcn_exp2f(-up);
            ref += up;
            above = seen || !first ? kLazy : kNothing;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DTILES; ++d)
                o[d] *= alpha;
            exponents();
        }
        half8_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = __builtin_amdgcn_exp2f(x[8 * j + e]);
                sum += y;
                p[j][e] = (_Float16)y; // to nearest: 2^-11 of a weight at most
            }
            l = fmaf(sum, g[j].z, l);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int d = 0; d < DTILES; ++d)
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lds.v[buf][(d * 4 + j) * 64 + (lane ^ (j << 1))], p[j], o[d], 0,
                                                              0, 0);
        if (more)
            store(buf ^ 1);
        __syncthreads();
    }

    // ---- rows to the output, through LDS for whole lines -------------------
    l = add_xor32(l);
    const float n = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t(*mine)[D + 8] = lds.out + wave * 32;
#pragma unroll
    for (int d = 0; d < DTILES; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<u32x2_t *>(&mine[col][d * 32 + 2 * i + 4 * h]) =
                (u32x2_t){Act<DT>::pack(o[d][i] * n, o[d][i + 1] * n), Act<DT>::pack(o[d][i + 2] * n, o[d][i + 3] * n)};
    __syncthreads();
    constexpr int LPR = D / 8; // lanes a row
#pragma unroll
    for (int i = 0; i < 32; i += 64 / LPR) {
        const int rr = i + lane / LPR, gr = row0 + wave * 32 + rr, d = (lane & (LPR - 1)) * 8;
        if (gr < s.rows) {
            const int ti = gr / a.group, th = kvh * a.group + gr - ti * a.group;
            *reinterpret_cast<u32x4_t *>(a.out + ((int64_t)(s.t0 + ti) * a.q_heads + th) * D + d) =
                *reinterpret_cast<const u32x4_t *>(&mine[rr][d]);
        }
    }
}

} // namespace

hipError_t launch_kv_prompt(const KvAttnArgs &a, int dtype, hipStream_t stream)
{
    const int row_blocks = (int)(((int64_t)a.max_new * a.group + kRows - 1) / kRows);
    const dim3 grid((unsigned)((int64_t)row_blocks * a.requests * a.kv_heads));
    if (a.head_dim == 64) {
        if (dtype == QW_F16)
            kv_prompt_kernel<64, QW_F16><<<grid, dim3(kThreads), 0, stream>>>(a, row_blocks);
        else
            kv_prompt_kernel<64, QW_BF16><<<grid, dim3(kThreads), 0, stream>>>(a, row_blocks);
    } else {
        if (dtype == QW_F16)
            kv_prompt_kernel<128, QW_F16><<<grid, dim3(kThreads), 0, stream>>>(a, row_blocks);
        else
            kv_prompt_kernel<128, QW_BF16><<<grid, dim3(kThreads), 0, stream>>>(a, row_blocks);
    }
    return hipGetLastError();
}

} // namespace qw
