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
// each wave in whole fragments of the matrix instruction: fragment f is 64
// pieces of 16 bytes, a lane's each, and a 65th place, so that the writes
// (eight lanes hold consecutive pieces of one row, that is of eight
// fragments) spread over the banks as the reads do.  Three buffers: the two
// waves of a SIMD take turns, one in the matrix phase (the values of a tile,
// the keys of the next) while the other is in the softmax phase, so that at
// the same time one tile is read, the next is written and a third is still
// read by the waves that come behind.  A barrier ends each phase.
//
// Bound by the phases' length.  By counters (eight chunks of 512 behind 15000, 32
// heads on 2: 512 workgroups of 242 tiles) a phase takes 1900 cycles, and a wave
// issues a tile 32 matrix instructions of 32 cycles, 1024 in all, and 200 vector
// ones, active for 920, beside 93 scalar and 40 LDS ones.  So one wave's products
// and the other's softmax take nearly as long as one behind the other: the matrix
// cores are busy 54 % of the time (42 % over prompts whose row blocks do not come
// out even).  Why the two overlap so little has not been found.  The staging of
// the next tile goes with the matrix phase (with the other one: 2 to 3 %
// slower; dealt out among the matrix instructions by hand: 15 % slower).
// Measured: four prompts of up to 8192 tokens, 32 query heads on 8 key heads,
// causal: 1080 us, 970 TFLOP/s fp16, and 1050 us in bf16 with blocks of 16 (a
// matrix product of 8192^3: 1151 and 1218); three of up to 4096 on 2 key heads
// 290 us, 870 TFLOP/s, where the row blocks do not come out even over the CUs.
// The form before this one (all waves in step, two buffers, staging with
// branches) took 2147 us for the first.
#include "kv_attention_device.h"

namespace qw {

namespace {

constexpr int D = 128;
constexpr int STEPS = D / 16; // of the first product
constexpr int DTILES = D / 32;
constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves; // query rows of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 64;
constexpr int kSlots = 65; // of a fragment: a lane each, and one so that fragments begin at different banks
constexpr int kAhead = 4; // fragments read ahead of the matrix instructions
constexpr int kSegment = 64; // tiles whose scales are fetched at once
constexpr int kFirst = 3; // number of the first tile: its buffers have index 0 (modulo 3)

union PromptLds {
    struct {
        half8_t k[3][D / 8][kSlots]; // [32-key half][16-channel step][lane]
        half8_t v[3][D / 8][kSlots]; // [32-channel tile][16-key step][lane]
        // per 16 keys: key scale * log2(e) * softmax scale, log2 of the value
        // scale, its inverse; of two segments of the keys
        float4_t scale[2][kSegment * 4];
    };
    uint16_t out[kRows][D + 8];
    struct {
        int sums[kWaves], found[2];
    };
};

template <int DT>
__global__ __launch_bounds__(kThreads, 2) void kv_prompt_kernel(KvAttnArgs a)
{
    __shared__ __attribute__((aligned(16))) PromptLds lds;

    const int tid = threadIdx.x, lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;
    // Which request and row block.  Workgroups that have nothing to do would
    // hold up the dispatch (each waits for a CU's LDS, and workgroups go round
    // the shader engines whatever they hold: with one long request among four,
    // 64 of 256 CUs worked), so the row blocks of all requests lie in a row, and
    // the host bounds their number by the tokens'.  Tokens of no request come behind,
    // if their rows are to be zeroed, as requests without keys.
    const int target = (int)blockIdx.x / a.kv_heads;
    const int kvh = (int)blockIdx.x - target * a.kv_heads;
    auto request = [&](int r) { return r < a.requests ? kv_request(a, r) : kv_gap(a, r - a.requests); };
    int r, row_block;
    if (!kv_find_block<kWaves>(a.requests + (a.zero_rest ? 2 : 0), kRows, [&](int i) { return request(i).rows; }, target, lds.sums,
                               lds.found, r, row_block))
        return; // (the bound's slack)
    const int row0 = row_block * kRows;
    const KvRequest s = request(r);
    __syncthreads(); // lds is the tiles' from here on
    const int last_row = row0 + kRows < s.rows ? row0 + kRows - 1 : s.rows - 1;
    const int first_i = row0 / a.group, last_i = last_row / a.group;
    // keys that some row of the block sees, and keys that every one does
    const int end = a.causal ? kv_clamp(s.past + last_i + 1, 0, s.ctx) : s.ctx;
    const int begin = a.window ? kv_clamp(s.past + first_i - a.window + 1, 0, end) & ~(kTile - 1) : 0;
    const int all_hi = a.causal ? s.past + first_i + 1 : s.ctx;
    const int all_lo = a.window ? s.past + last_i - a.window + 1 : 0;

    // ---- staging: what this thread brings into LDS -------------------------
    // A piece of 16 bytes of each: 16 channels of a key (kt, kc) and 16 keys of
    // a channel (vd, vk).  They are dealt out so that a wave's pieces of a tile
    // lie in one block, whatever the block size: its address is scalar work, and
    // a lane's offset in the block never changes.  Keys are fetched a tile ahead
    // of the values.  The staging has no branches: the compiler could not count
    // the loads in flight across them, and would wait for all (1000 cycles a
    // tile).
    const int shift = a.block_shift, block = 1 << shift;
    const int64_t head_bytes = (int64_t)block * D;
    const int32_t *table = a.block_table + (int64_t)r * a.table_width;
    static_assert(kTile * D / 16 == kThreads, "a piece of each operand a thread");
    const int side = shift < 6 ? shift - 4 : 2; // log2 of a block's pieces of one channel, of a tile
    const int kt = tid / (D / 16), kc = tid % (D / 16);
    const int vb = tid >> side >> 7, vd = (tid >> side) & (D - 1), vk = (tid & ((1 << side) - 1)) + (vb << side);
    const uint32_t k_at = (uint32_t)((kt & (block - 1)) * D + kc * 16), v_at = (uint32_t)(vd * block + ((vk * 16) & (block - 1)));
    const int k_first = __builtin_amdgcn_readfirstlane(kt & ~15), v_first = __builtin_amdgcn_readfirstlane((vb << side) * 16);
    // row m of the first product's tile holds key u of 32
    const int u = kt & 31, m = (u & 3) + 16 * (u >> 4) + 8 * ((u >> 2) & 1) + 4 * ((u >> 3) & 1);
    auto known = [&](int32_t id) { return id >= 0 && id < a.num_blocks; };
    auto row_of = [&](int32_t id) { return (int64_t)(known(id) ? id : 0) * a.kv_heads + kvh; };
    // The block of key j (of the last key, behind it: read and masked).
    auto look = [&](int j) { return table[(j < end ? j : end - 1) >> shift]; };
    u32x4_t kraw, vraw;
    int32_t kid, vid; // blocks of the next pieces
    auto look_k = [&](int base) { kid = look(base + k_first); };
    auto look_v = [&](int base) { vid = look(base + v_first); };
    auto fetch_k = [&](int base) {
        kraw = *reinterpret_cast<const u32x4_t *>(a.k_cache + row_of(__builtin_amdgcn_readfirstlane(kid)) * head_bytes +
                                                  (base & (block - 1)) * D + k_at);
    };
    auto fetch_v = [&](int base) {
        vraw = *reinterpret_cast<const u32x4_t *>(a.v_cache + row_of(__builtin_amdgcn_readfirstlane(vid)) * head_bytes +
                                                  (base & (block - 1)) + v_at);
    };
    auto put_k = [&](int tile) {
        half8_t *at = &lds.k[tile % 3][(kt >> 5) * STEPS + kc][m];
        at[0] = i8x8_to_half8(kraw.x, kraw.y);
        at[32] = i8x8_to_half8(kraw.z, kraw.w);
    };
    auto put_v = [&](int tile) {
        half8_t *at = &lds.v[tile % 3][(vd >> 5) * 4 + vk][vd & 31];
        at[0] = i8x8_to_half8(vraw.x, vraw.y);
        at[32] = i8x8_to_half8(vraw.z, vraw.w);
    };
    // The scales of a segment, one 16-key group a thread: log2 and inverse once,
    // not by every wave for every tile.  Groups behind the last key get its
    // block's: their weights are 0, and 0 has to be multiplied by a finite inverse.
    auto segment_scales = [&](int segment) {
        if (tid < kSegment * 4) {
            const int32_t at = look(begin + segment * (kSegment * kTile) + tid * 16);
            const float ks = a.k_scales[row_of(at)], vs = fmaxf(a.v_scales[row_of(at)], kKvScaleFloor);
            // (a group without a block: scores of -inf, whatever its codes)
            lds.scale[segment & 1][tid] = known(at) ? (float4_t){ks * a.scale_log2, __builtin_amdgcn_logf(vs), 1.0f / vs, 0.0f}
                                                    : (float4_t){0.0f, -INFINITY, 0.0f, 0.0f};
        }
    };
    // Puts down the values of tile number `tile` (at key `base`) and the keys of
    // the next, and asks for what the next call puts down.
    auto stage = [&](int tile, int base) {
        put_k(tile + 1);
        put_v(tile);
        fetch_k(base + 2 * kTile);
        fetch_v(base + kTile);
        look_k(base + 3 * kTile);
        look_v(base + 2 * kTile);
    };

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
    float ref = 0.0f, l = 0.0f;
    bool seen = !in; // a key; both lanes of a row agree

    float16_t sc[2];
    half8_t p[4];
    // Matrix phase: the second product of a tile, and the first product of the
    // next.  Fragments are read kAhead before their use.  (The empty asm keeps a
    // buffer's address in one register, so that fragments are constant offsets
    // from it; folded into them it would leave the instruction's range.)
    typedef __attribute__((address_space(3))) const half8_t lds_half8;
    auto key_product = [&](int buf) {
        lds_half8 *k = (lds_half8 *)&lds.k[buf][0][lane];
        asm("" : "+v"(k));
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                sc[t][i] = 0.0f;
#pragma unroll
        for (int c = 0; c < STEPS; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t)
                sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[(t * STEPS + c) * kSlots], q[c], sc[t], 0, 0, 0);
    };
    auto value_product = [&](int buf) {
        lds_half8 *v = (lds_half8 *)&lds.v[buf][0][lane];
        asm("" : "+v"(v));
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int d = 0; d < DTILES; ++d)
                o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[(d * 4 + j) * kSlots], p[j], o[d], 0, 0, 0);
    };
    auto order = [&]() {
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0); // LDS reads
#pragma unroll
        for (int i = 0; i < 4 * DTILES + 2 * STEPS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0); // a matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
    };
    // Softmax phase: the weights of a tile.  A row's reference moves when its
    // weights get large (their sum tells, without a maximum over them), and at
    // the first tile of which the row sees a key.
    float4_t g[4]; // the tile's scales, read while the matrix instructions run
    auto read_scales = [&](int tile) {
        const int n = tile - kFirst;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            g[j] = lds.scale[n / kSegment & 1][(n & (kSegment - 1)) * 4 + j];
    };
    auto softmax = [&](int base) {
        float inv[4], sum[4], y[32];
        // scores become exponents relative to the reference (8 scores of a lane
        // share a scale)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c = g[j].x * down, b = g[j].y - ref;
            inv[j] = g[j].z;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sc[j >> 1][(j & 1) * 8 + e] = fmaf(sc[j >> 1][(j & 1) * 8 + e], c, b);
        }
        if (base < all_lo || base + kTile > all_hi) {
            const int lo = lim_lo - base - h * 8, hi = lim_hi - base - h * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j * 16 + e < lo || j * 16 + e >= hi)
                        sc[j >> 1][(j & 1) * 8 + e] = -INFINITY;
        }
        auto weights = [&]() {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum[j] = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[8 * j + e] = __builtin_amdgcn_exp2f(sc[j >> 1][(j & 1) * 8 + e]);
                    sum[j] += y[8 * j + e];
                }
            }
        };
        weights();
        float most = fmaxf(fmaxf(sum[0], sum[1]), fmaxf(sum[2], sum[3]));
        if (__any(!seen || most >= kKvLarge)) {
            // (a row moves for its own sake only: no result depends on which rows
            // share a wave)
            most = max_xor32(most);
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top = fmaxf(top, sc[t][i]);
            top = max_xor32(top);
            const float up = (seen ? most >= kKvLarge : top > kKvNothing) ? top - kKvRise : 0.0f; // the new reference lies so far above the old
            const float alpha = seen ? __builtin_amdgcn_exp2f(-up) : 1.0f;
            ref += up;
            seen = seen || top > kKvNothing;
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DTILES; ++d)
                o[d] *= alpha;
            sc[0] -= up;
            sc[1] -= up;
            weights();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            l = fmaf(sum[j], inv[j], l);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                p[j][e] = (_Float16)y[8 * j + e]; // to nearest (the error: see kKvRise)
        }
    };

    // The first two tiles' keys, the first one's values; what follows is asked
    // for.
    if (begin < end) {
        look_k(begin);
        look_v(begin);
        fetch_k(begin);
        look_k(begin + kTile);
        put_k(kFirst);
        fetch_k(begin + kTile);
        fetch_v(begin);
        look_k(begin + 2 * kTile);
        look_v(begin + kTile);
        segment_scales(0);
        stage(kFirst, begin);
    }
    __syncthreads();

    // While waves 0 to 3 are in the softmax phase of a tile, waves 4 to 7 are in
    // the matrix phase before it, and the other way round.  With a phase's number
    // behind a barrier, the first waves' matrix phase of tile n is 2 n + 1, the
    // others' 2 n + 2.  In it they put down the keys of tile n + 2 and the values
    // of n + 1, which are read from phase 2 n + 3 on, in the place of keys n - 1
    // and values n - 2, which were read in phase 2 n - 2 at the latest.
    const bool second = wave >= 4;
    if (second)
        __syncthreads();
    key_product(kFirst % 3);
    read_scales(kFirst);
    __syncthreads();
    int tile = kFirst;
    for (int base = begin; base < end; base += kTile, ++tile) {
        softmax(base);
        if (((tile - kFirst) & (kSegment - 1)) == kSegment / 2)
            segment_scales((tile - kFirst) / kSegment + 1);
        __syncthreads();
        __builtin_amdgcn_s_setprio(1);
        stage(tile + 1, base + kTile);
        value_product(tile % 3);
        key_product((tile + 1) % 3); // (behind the last tile: not used)
        order();
        read_scales(tile + 1);
        __builtin_amdgcn_s_setprio(0);
        __syncthreads();
    }
    if (!second)
        __syncthreads();

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
    // row blocks of all requests: full ones of the tokens' rows, and a last one each
    const int64_t each = ((int64_t)a.max_new * a.group + kRows - 1) / kRows * a.requests;
    const int64_t full = (int64_t)a.tokens * a.group / kRows + a.requests;
    const dim3 grid((unsigned)((a.zero_rest ? full + 2 : each < full ? each : full) * a.kv_heads));
    if (dtype == QW_F16)
        kv_prompt_kernel<QW_F16><<<grid, dim3(kThreads), 0, stream>>>(a);
    else
        kv_prompt_kernel<QW_BF16><<<grid, dim3(kThreads), 0, stream>>>(a);
    return hipGetLastError();
}

} // namespace qw
