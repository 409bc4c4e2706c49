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
//   t_j = log2(e) s_j + log2 Sv(j),  P_j = 2^{t_j - M}
//   o = sum P_j Vq[j] / sum (P_j / Sv(j))
// so one running reference M serves both sums, whatever the scales of the
// blocks, and the denominator needs one multiplication per 16 keys.  M lies
// 8 below the maximum of the first tile in which the row sees a key, and moves
// to a later tile's only where weights of that one add up to 2^16 (a sum that is
// there anyway: no maximum is taken over the other tiles); the accumulators
// are rescaled then.  So P stays below fp16's range, and some P is 2^8 or
// more.  M, the denominators and the accumulators are fp32.
//
// Query rows that share a key head (the heads of its group, for each new
// token) form the columns of one matrix product, so the cache is read once
// for all of them.
#include "kv_attention_device.h"

namespace qw {

namespace {

constexpr int kThreads = 256; // of the join
constexpr int kTile = 64; // keys a wave takes at once
// What beginning and ending a unit costs a workgroup, in tiles: a workgroup
// whose range spans several units is given fewer keys.  (0, 4 and 8: 34.3,
// 32.9 and 33.4 us for 64 requests of 512 to 8192 keys, 38.0, 28.0 and 28.3 us
// for 48 of 128 to 2048 with 16 key heads.)
constexpr int kUnitCost = 4;
constexpr int kMinRange = 4 + kUnitCost; // of a workgroup's range, at least

constexpr int kWaves = 4; // of a split workgroup

// Tiles in one workgroup that are worth two more launches (see attn_plan): some
// 70 us of the prompt kernel, at 2.3 a tile, or of the split kernel, at 0.5.
// There a quarter of that where most workgroups find no rows: they pass through
// what slots the long ones leave (64 requests, one of 512 tokens and the others
// of one behind 8000: 451 us and 62).  (32 always: eight windowed chunks of 64
// channels, up to 72 tiles and half of the workgroups empty, 96 us for 91.)
constexpr int long_walk(bool prompt, bool sparse) { return prompt || sparse ? 32 : 128; }

// Ranges a CU.  Two keep its memory pipe full where a tile is 16 KiB; with
// tiles of 8 KiB and one row tile three do better (24.9 us against 28.0 for
// 48 requests of 128 to 2048 keys, 16 key heads of 64 channels), while at 128
// channels three are slower (33.2 against 32.9 us for 64 requests of 512 to
// 8192 keys; 95 against 74 us with two row tiles): the older workgroups of a
// CU are served first, and the youngest ends alone.
constexpr int split_groups(int head_dim, int row_tiles) { return head_dim == 64 && row_tiles == 1 ? 3 : 2; }

// Where the 64 keys of a tile lie.
enum Layout {
    kNarrow = 0, // in several blocks
    kWhole = 1,  // in one block of 64
    kHalf = 2    // in one block of 128: a value row of the tile is half a cache line
};

// A request, with the keys that any of its rows sees and their cost.
struct Request : KvRequest {
    int lo, hi; // keys; lo is a multiple of kTile
    int cost;   // of a unit: kTile-key tiles of that range, at least one, and kUnitCost; 0 without rows

    // of all its units: those of each key head and block of 16 RT query rows
    template <int RT>
    __device__ __forceinline__ int total(const KvAttnArgs &a) const { return cost * ((rows + 16 * RT - 1) / (16 * RT) * a.kv_heads); }
};

__device__ __forceinline__ Request request_of(const KvAttnArgs &a, int r)
{
    Request s;
    static_cast<KvRequest &>(s) = kv_request(a, r);
    s.lo = s.hi = 0;
    s.cost = 0;
    if (s.rows) {
        s.hi = a.causal ? kv_clamp(s.past + s.rows / a.group, 0, s.ctx) : s.ctx;
        s.lo = a.window ? kv_clamp(s.past - a.window + 1, 0, s.hi) & ~(kTile - 1) : 0;
        s.cost = (s.hi > s.lo ? (s.hi - s.lo + kTile - 1) / kTile : 1) + kUnitCost;
    }
    return s;
}

// The same, and behind the requests the tokens of none, whose rows see no key.
__device__ __forceinline__ Request request_or_gap(const KvAttnArgs &a, int r)
{
    if (r < a.requests)
        return request_of(a, r);
    Request s;
    static_cast<KvRequest &>(s) = kv_gap(a, r - a.requests);
    s.lo = s.hi = 0;
    s.cost = s.rows ? 1 + kUnitCost : 0;
    return s;
}

// ---------------------------------------------------------------------------
// Split kernel: the 64-key tiles of a unit (one key head and block of 16 RT
// query rows of one request) are taken in turn by the waves of a workgroup,
// which are joined through LDS at the end of the unit.
//
// S^T = Kq Q^T and O^T = Vq^T P^T on v_mfma_f32_16x16x32_f16.  A lane holds
// column (query row) lane & 15 of S^T; which keys its registers hold depends
// only on which cache rows fed the first product, and they are chosen so
// that lane group g = lane / 16 holds keys 16 g .. 16 g + 15 of the tile:
// exactly the operand layout of the second product, whose other operand is
// then one contiguous 16-byte load a lane from the transposed values.
// Nothing passes through LDS or between lanes until the unit's end, but a row's
// maximum where its reference moves.
//
// Bound by HBM: 2 * D + 8 / B bytes a key and head, read straight into
// registers; past the caches where there is one block of query rows (ONCE:
// 6.0 against 5.6 TB/s on long contexts), else through them (64 tokens behind
// 131072, 32 heads on 2: 260 us for 350; eight prompts of 4096, 16 heads of 64:
// 465 for 510).  A
// tile is D / 4 loads of 16 bytes a lane in flight; asking for the next tile
// before this one's products gained nothing, with eight waves a CU.
// ---------------------------------------------------------------------------
template <int D, int RT>
struct SplitLds {
    float o[kWaves][16 * RT][D + 4];
    float m[kWaves][16 * RT], l[kWaves][16 * RT];
};

// Codes that are read once bypass the caches.
template <bool ONCE>
__device__ __forceinline__ u32x4_t load_codes(const int8_t *p)
{
    const u32x4_t *at = reinterpret_cast<const u32x4_t *>(p);
    return ONCE ? __builtin_nontemporal_load(at) : *at;
}

// Floats of an unfinished piece in the workspace: 16 RT rows of D channels,
// the reference M, the denominator, and two of padding.
constexpr int piece_floats(int head_dim, int row_tiles) { return 16 * row_tiles * (head_dim + 4); }

// Tiles of one unit.
struct Piece {
    Request s;
    int r, kvh, row0;
    int begin, end; // keys
    float *part;    // where it is left unfinished; null: it is the whole unit
};

// What the join has to know of a unit in several ranges.
struct Cut {
    int kvh, row0;
    int first, last; // ranges that hold tiles of it
    int slot;        // which of the first one's two pieces is its own
    int t0, rows;
};

// A workgroup's range, handed out piece by piece.  The units of all requests
// lie in a row, request by request, each as long as its cost: kUnitCost, then
// its tiles.
struct Range {
    int begin, at, stop;
    Request s;   // request r; the requests before it cost `before`
    int r, before;
    float *parts; // room for two pieces: one at the range's begin, one at its end

    // `cut` (may be null) is told of the unit that begins here and goes on
    // behind the range.
    template <int D, int RT>
    __device__ __forceinline__ bool next(const KvAttnArgs &a, Piece &p, Cut *cut)
    {
        while (at < stop) {
            const int behind = before + s.template total<RT>(a);
            if (at >= behind) {
                before = behind;
                s = request_or_gap(a, ++r);
                continue;
            }
            const int rel = at - before;
            const int unit = rel / s.cost, from = rel - unit * s.cost;
            const int count = s.cost - from < stop - at ? s.cost - from : stop - at;
            const int off = from > kUnitCost ? from - kUnitCost : 0, tiles = from + count - kUnitCost - off;
            const int rb = unit / a.kv_heads;
            p.s = s;
            p.r = r;
            p.kvh = unit - rb * a.kv_heads;
            p.row0 = rb * 16 * RT;
            p.begin = s.lo + off * kTile;
            p.end = s.hi - p.begin < tiles * kTile ? s.hi : p.begin + tiles * kTile;
            const bool leads = at == begin;
            p.part = tiles == s.cost - kUnitCost ? nullptr : (leads ? parts : parts + piece_floats(D, RT));
            at += count;
            if (tiles > 0) {
                if (p.part && off == 0 && cut) { // (so this is not the last range, and as long as all but that)
                    const int last = (before + (unit + 1) * s.cost - 1) / (stop - begin);
                    if (threadIdx.x == 0)
                        *cut = {p.kvh, p.row0, (int)blockIdx.x, last, leads ? 0 : 1, s.t0, s.rows};
                }
                return true;
            }
        }
        return false;
    }
};

template <int D, int RT, int DT, int LAYOUT, bool ONCE>
__device__ __forceinline__ void split_piece(const KvAttnArgs &a, const Piece &p, SplitLds<D, RT> &lds)
{
    constexpr int CH = D / 64; // 64-channel pieces of a key row
    constexpr int DTILES = D / 16;
    constexpr int NW = kWaves;

    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int shift = LAYOUT == kWhole ? 6 : (LAYOUT == kHalf ? 7 : a.block_shift);
    const int block = 1 << shift;
    const int64_t head_bytes = (int64_t)block * D;

    // query rows, as the first product's second operand
    half8_t q[RT][CH][2];
    float mult[RT]; // scores -> exponents of 2, without the key scale
    int lim_lo[RT], lim_hi[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = p.row0 + t * 16 + col;
        const bool in = row < p.s.rows;
        const int i = in ? row / a.group : 0, head = p.kvh * a.group + (in ? row - i * a.group : 0);
        const uint16_t *src = a.q + (int64_t)(p.s.t0 + i) * a.q_stride + (int64_t)head * D + g * 16;
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
            kv_row_power(max_xor32(max_xor16(top)), up, down);
        mult[t] = a.scale_log2 * down;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                q[t][c][h] = kv_half8<DT>(raw[c][h], up);
        lim_hi[t] = in ? (a.causal ? p.s.past + i + 1 : p.s.ctx) : 0;
        lim_lo[t] = a.window ? p.s.past + i - a.window + 1 : 0;
    }
    // keys that every row of the block sees
    const int last_row = p.row0 + 16 * RT < p.s.rows ? p.row0 + 16 * RT - 1 : p.s.rows - 1;
    const int all_hi = a.causal ? p.s.past + p.row0 / a.group + 1 : p.s.ctx;
    const int all_lo = a.window ? p.s.past + last_row / a.group - a.window + 1 : 0;
    // keys that some row of the block sees, of the piece's
    const int any_hi = a.causal ? p.s.past + last_row / a.group + 1 : p.s.ctx;
    const int any_lo = a.window ? (p.s.past + p.row0 / a.group - a.window + 1) & ~(kTile - 1) : 0;
    const int begin = p.begin > any_lo ? p.begin : any_lo, end = p.end < any_hi ? p.end : any_hi;

    float4_t o[RT][DTILES];
    float m[RT], l[RT]; // the reference, and the denominator over this lane's keys
    bool seen[RT];      // a key; the four lanes of a row agree
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        m[t] = 0.0f;
        seen[t] = p.row0 + t * 16 + col >= p.s.rows;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
            o[t][d] = (float4_t){0, 0, 0, 0};
    }

    const int32_t *table = a.block_table + (int64_t)p.r * a.table_width;
    // Cache row (block and head) that holds key j; block 0's where the table
    // holds none: it is read in its place and masked.
    auto row_of = [&](int j, bool &ok) {
        const int32_t id = j < end ? table[j >> shift] : -1;
        ok = id >= 0 && id < a.num_blocks;
        return (int64_t)(ok ? id : 0) * a.kv_heads + p.kvh;
    };

    for (int base = begin + wave * kTile; base < end; base += NW * kTile) {
        // Key rows: row c of 16-key product i is key 16 (c / 4) + 4 i + c % 4.
        u32x4_t kraw[4][CH], vraw[DTILES];
        bool ok;
        int64_t kb, vb;
        if (LAYOUT != kNarrow) {
            kb = vb = row_of(base, ok);
        } else {
            bool unused;
            kb = row_of(base + (col >> 2) * 16, unused);
            vb = row_of(base + g * 16, ok);
        }
        const uint32_t k_at = (uint32_t)(((base + (col >> 2) * 16) & (block - 1)) + (col & 3)) * D + g * 16;
        const uint32_t v_at = (uint32_t)(col * block + ((base + g * 16) & (block - 1)));
        const int8_t *kp = a.k_cache + kb * head_bytes + k_at;
        const int8_t *vp = a.v_cache + vb * head_bytes + v_at;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                kraw[i][c] = load_codes<ONCE>(kp + i * 4 * D + c * 64);
        const float ks = a.k_scales[vb], vs = a.v_scales[vb];
#pragma unroll
        for (int d = 0; d < DTILES; ++d) // (of a half line the other half follows)
            vraw[d] = load_codes<ONCE && LAYOUT != kHalf>(vp + d * 16 * block);

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
        half8_t w[RT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const float c = ok ? mult[t] * ks : 0.0f, b = lv - m[t];
            float x[16], y[16], sum;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[4 * i + j] = fmaf(sc[t][i][j], c, b);
            if (!whole) {
                const int at = base + g * 16;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = ok && at + e >= lim_lo[t] && at + e < lim_hi[t] ? x[e] : -INFINITY;
            }
            auto weights = [&]() {
                sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    y[e] = __builtin_amdgcn_exp2f(x[e]);
                    sum += y[e];
                }
            };
            weights();
            if (__any(!seen[t] || sum >= kKvLarge)) {
                // (a row moves for its own sake only: no result depends on which
                // rows share a wave)
                const float most = max_xor32(max_xor16(sum));
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    top = fmaxf(top, x[e]);
                top = max_xor32(max_xor16(top));
                const float up = (seen[t] ? most >= kKvLarge : top > kKvNothing) ? top - kKvRise : 0.0f;
                const float alpha = seen[t] ? __builtin_amdgcn_exp2f(-up) : 1.0f;
                m[t] += up;
                seen[t] = seen[t] || top > kKvNothing;
                l[t] *= alpha;
#pragma unroll
                for (int d = 0; d < DTILES; ++d)
                    o[t][d] *= alpha;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] -= up;
                weights();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
                w[t][e >> 3][e & 7] = (_Float16)y[e]; // to nearest (the error: see kKvRise)
            l[t] = fmaf(sum, inv, l[t]);
        }
#pragma unroll
        for (int d = 0; d < DTILES; ++d) {
            const half8_t v0 = i8x8_to_half8(vraw[d].x, vraw[d].y);
            const half8_t v1 = i8x8_to_half8(vraw[d].z, vraw[d].w);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[t][0], o[t][d], 0, 0, 0);
                o[t][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[t][1], o[t][d], 0, 0, 0);
            }
        }
    }

    // join the waves
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] = add_xor32(add_xor16(l[t]));
        if (g == 0) {
            lds.m[wave][t * 16 + col] = seen[t] ? m[t] : -INFINITY;
            lds.l[wave][t * 16 + col] = l[t];
        }
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
            *reinterpret_cast<float4_t *>(&lds.o[wave][t * 16 + col][d * 16 + g * 4]) = o[t][d];
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        // 16 threads a row, E channels each
        constexpr int E = D / 16;
        const int row = t * 16 + ((int)threadIdx.x >> 4), d0 = ((int)threadIdx.x & 15) * E;
        float ref = lds.m[0][row];
#pragma unroll
        for (int w = 1; w < NW; ++w)
            ref = fmaxf(ref, lds.m[w][row]);
        float sum = 0.0f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float mw = lds.m[w][row];
            const float f = mw == ref ? 1.0f : __builtin_amdgcn_exp2f(mw - ref);
            sum = fmaf(lds.l[w][row], f, sum);
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] = fmaf(lds.o[w][row][d0 + e], f, acc[e]);
        }
        const int gr = p.row0 + row;
        if (gr < p.s.rows) {
            if (!p.part) {
                const int i = gr / a.group, head = p.kvh * a.group + gr - i * a.group;
                const float n = sum == 0.0f ? 0.0f : 1.0f / sum;
                uint16_t *out = a.out + ((int64_t)(p.s.t0 + i) * a.q_heads + head) * D + d0;
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<uint32_t *>(out + e) = Act<DT>::pack(acc[e] * n, acc[e + 1] * n);
            } else {
                float *w = p.part + row * (D + 4);
#pragma unroll
                for (int e = 0; e < E; e += 4)
                    *reinterpret_cast<float4_t *>(w + d0 + e) = (float4_t){acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
                if (d0 == 0) {
                    w[D] = ref;
                    w[D + 1] = sum;
                }
            }
        }
    }
    __syncthreads();
}

// Zeroes the rows of no request, where that is asked for: by the first workgroups
// of the unit form, when their own work is done (by all of them, when they begin:
// 264 us for 248 for eight prompts of up to 4096 with 64 channels, 104 for 91 for
// 1024 single tokens).
__device__ __forceinline__ void zero_rest(const KvAttnArgs &a)
{
    const unsigned group = blockIdx.y * gridDim.x + blockIdx.x, all = gridDim.x * gridDim.y, groups = all < 256 ? all : 256;
    if (!a.zero_rest || group >= groups)
        return;
    const int64_t row = (int64_t)a.q_heads * a.head_dim;
    for (int g = 0; g < 2; ++g) {
        const KvRequest s = kv_gap(a, g);
        for (int64_t t = group; t < -s.past; t += groups)
            for (int64_t i = threadIdx.x * 8; i < row; i += blockDim.x * 8)
                *reinterpret_cast<u32x4_t *>(a.out + (s.t0 + t) * row + i) = (u32x4_t){0, 0, 0, 0};
    }
}

// One workgroup a unit: for contexts that one workgroup reads fast enough,
// or units enough to fill the chip many times over.  The grid is units and
// requests, or (`dense`) the row blocks that there are at most: where the
// requests' numbers of rows differ much most workgroups of the first find none,
// at 1 ns each (one prompt of 4096 beside 255 tokens, 16 heads of 64, behind
// 500: 529 us and 125; 1024 single tokens, all of them there, 91 and 95).
template <int D, int RT, int DT, int LAYOUT, bool ONCE>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_unit_kernel(KvAttnArgs a, bool dense)
{
    __shared__ __attribute__((aligned(16))) SplitLds<D, RT> lds;
    __shared__ int sums[kWaves], found[2];
    int rb = (int)blockIdx.x / a.kv_heads, r = blockIdx.y;
    const int kvh = (int)blockIdx.x - rb * a.kv_heads;
    bool any = true;
    if (dense)
        any = kv_find_block<kWaves>(a.requests, 16 * RT, [&](int i) { return kv_request(a, i).rows; }, rb, sums, found, r, rb);
    if (any) {
        const Request s = request_of(a, r);
        const Piece p = {s, r, kvh, rb * 16 * RT, s.lo, s.hi, nullptr};
        if (p.row0 < s.rows)
            split_piece<D, RT, DT, LAYOUT, ONCE>(a, p, lds);
    }
    zero_rest(a);
}

// The tiles of all units in a row, cut into equal ranges, split_groups a CU:
// every workgroup streams the same number of keys, whatever the requests' numbers
// of keys and of query rows and however far the host's bounds are above them.  A
// unit that lies in one range is written out; the others' pieces (a range has
// two at most: where it begins and where it ends) go to the workspace and are
// joined by a second kernel.
//
// Workspace: for a join by requests the ranges' length, the cost before each
// request and that of its units (int32, 2 requests + 1 of them), for a join by
// ranges a Cut a range; from the next multiple of four words on, two pieces a
// range.
__device__ __host__ __forceinline__ int64_t parts_offset(int64_t requests, int64_t groups)
{
    const int64_t cuts = groups * (int64_t)(sizeof(Cut) / sizeof(int32_t));
    return ((cuts > 2 * requests + 1 ? cuts : 2 * requests + 1) + 3) / 4 * 4;
}

template <int D, int RT, int DT, int LAYOUT, bool ONCE>
__global__ __launch_bounds__(64 * kWaves, 2) void kv_stream_kernel(KvAttnArgs a, bool by_ranges)
{
    constexpr int NW = kWaves, NT = 64 * NW;
    __shared__ __attribute__((aligned(16))) SplitLds<D, RT> lds;
    __shared__ int wave_sums[NW];
    __shared__ Request found; // the request that holds the range's first tile,
    __shared__ int found_r, found_before; // its number and the cost before it
    const int lane = __lane_id(), wave = (int)threadIdx.x >> 6;
    int32_t *head = reinterpret_cast<int32_t *>(a.workspace);
    Cut *cuts = reinterpret_cast<Cut *>(a.workspace);

    const int requests = a.requests + (a.zero_rest ? 2 : 0); // with the gaps

    // Cost before each request of a batch of NT; `sum` grows by the batch's.
    auto scan = [&](int cost, int &sum) {
        int upto = cost;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(upto, d);
            upto += lane >= d ? up : 0;
        }
        if (lane == 63)
            wave_sums[wave] = upto;
        __syncthreads();
        int before = sum + upto - cost;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            before += w < wave ? wave_sums[w] : 0;
            sum += wave_sums[w];
        }
        return before;
    };
    auto batch = [&](int r) {
        Request s = request_or_gap(a, r < requests ? r : requests - 1);
        s.cost = r < requests ? s.cost : 0;
        return s;
    };

    int total = 0, before = 0;
    Request mine;
    for (int base = 0; base < requests; base += NT) {
        if (base)
            __syncthreads(); // wave_sums has been read
        const int r = base + (int)threadIdx.x;
        mine = batch(r);
        before = scan(mine.template total<RT>(a), total);
        if (!by_ranges && blockIdx.x == 0 && r < a.requests) {
            head[1 + 2 * r] = before;
            head[2 + 2 * r] = mine.cost;
        }
    }
    int per = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    per = per < kMinRange ? kMinRange : per;
    if (by_ranges && threadIdx.x == 0)
        cuts[blockIdx.x] = {0, 0, 0, -1, 0, 0, 0};
    if (!by_ranges && blockIdx.x == 0 && threadIdx.x == 0)
        head[0] = per;
    Range range;
    range.begin = range.at = (int)blockIdx.x * per;
    if (range.at >= total)
        return;
    range.stop = total - range.at < per ? total : range.at + per;
    range.parts = a.workspace + parts_offset(a.requests, gridDim.x) + (int64_t)blockIdx.x * 2 * piece_floats(D, RT);
    const int first = range.at;
    int sum = 0;
    for (int base = 0; base < requests; base += NT) {
        const int r = base + (int)threadIdx.x;
        if (requests > NT) { // once more, batch by batch
            __syncthreads();
            mine = batch(r);
            before = scan(mine.template total<RT>(a), sum);
        }
        if (before <= first && first < before + mine.template total<RT>(a)) {
            found = mine;
            found_r = r;
            found_before = before;
        }
        if (first < sum)
            break;
    }
    __syncthreads();
    range.r = __builtin_amdgcn_readfirstlane(found_r);
    range.before = __builtin_amdgcn_readfirstlane(found_before);
    range.s.t0 = __builtin_amdgcn_readfirstlane(found.t0);
    range.s.past = __builtin_amdgcn_readfirstlane(found.past);
    range.s.ctx = __builtin_amdgcn_readfirstlane(found.ctx);
    range.s.rows = __builtin_amdgcn_readfirstlane(found.rows);
    range.s.lo = __builtin_amdgcn_readfirstlane(found.lo);
    range.s.hi = __builtin_amdgcn_readfirstlane(found.hi);
    range.s.cost = __builtin_amdgcn_readfirstlane(found.cost);
    Piece p;
    while (range.template next<D, RT>(a, p, by_ranges ? cuts + blockIdx.x : nullptr))
        split_piece<D, RT, DT, LAYOUT, ONCE>(a, p, lds);
}

// Joins the pieces of a row: a workgroup for each row, its four waves over the
// pieces, their lanes over the channels.  By requests (the grid is rows, key
// heads, requests), or where these are too many, most of them empty because
// the requests' numbers of rows differ, by ranges (those, and the rows of a unit),
// the unit that is cut at the range's end being the workgroup's.
template <int D, int RT, int DT, bool BY_RANGES>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(KvAttnArgs a, int groups)
{
    constexpr int E = D / 64;
    __shared__ float lds[4][64 * E + 2];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    Cut cut;
    int row;
    if (BY_RANGES) {
        cut = reinterpret_cast<const Cut *>(a.workspace)[blockIdx.x];
        row = cut.row0 + (int)blockIdx.y;
        if (cut.last < 0 || row >= cut.rows)
            return;
    } else {
        const int32_t *head = reinterpret_cast<const int32_t *>(a.workspace);
        const int r = blockIdx.z, per = head[0], before = head[1 + 2 * r], cost = head[2 + 2 * r];
        const KvRequest s = kv_request(a, r);
        row = blockIdx.x;
        if (row >= s.rows)
            return;
        const int rb = row / (16 * RT), at = before + (rb * a.kv_heads + (int)blockIdx.y) * cost; // where the unit begins
        cut = {(int)blockIdx.y, rb * 16 * RT, (at + kUnitCost) / per, (at + cost - 1) / per, 0, s.t0, s.rows};
        if (cut.first == cut.last)
            return; // written by its only workgroup
        cut.slot = at > cut.first * per; // behind the end of another unit, else first in its range
    }
    const int first = cut.first;
    constexpr int64_t piece = piece_floats(D, RT);
    const float *parts = a.workspace + parts_offset(a.requests, groups) + (row - cut.row0) * (D + 4);
    auto part_of = [&](int w) { return parts + ((int64_t)w * 2 + (w == first ? cut.slot : 0)) * piece; };
    float m = -INFINITY, l = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.0f;
#pragma unroll 4
    for (int w = first + wave; w <= cut.last; w += 4) {
        const float *p = part_of(w);
        const float pm = p[D], pl = p[D + 1];
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            v[e] = p[lane * E + e];
        const float next = fmaxf(m, pm);
        const float fa = m == next ? 1.0f : __builtin_amdgcn_exp2f(m - next);
        const float fb = pm == next ? 1.0f : __builtin_amdgcn_exp2f(pm - next);
        m = next;
        l = l * fa + pl * fb;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * fa + v[e] * fb;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        lds[wave][lane * E + e] = acc[e];
    if (lane == 0) {
        lds[wave][64 * E] = m;
        lds[wave][64 * E + 1] = l;
    }
    __syncthreads();
    if (wave)
        return;
    float ref = lds[0][64 * E];
#pragma unroll
    for (int w = 1; w < 4; ++w)
        ref = fmaxf(ref, lds[w][64 * E]);
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float mw = lds[w][64 * E];
        const float f = mw == ref ? 1.0f : __builtin_amdgcn_exp2f(mw - ref);
        l += lds[w][64 * E + 1] * f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] += lds[w][lane * E + e] * f;
    }
    const float n = l == 0.0f ? 0.0f : 1.0f / l;
    const int i = row / a.group, qh = cut.kvh * a.group + row - i * a.group;
    uint16_t *out = a.out + ((int64_t)(cut.t0 + i) * a.q_heads + qh) * D + lane * E;
    if (E == 2)
        *reinterpret_cast<uint32_t *>(out) = Act<DT>::pack(acc[0] * n, acc[E - 1] * n);
    else
        *out = (uint16_t)Act<DT>::pack(acc[0] * n, 0.0f);
}

// Tiles that a row's workgroup may have to go through.
int64_t longest_walk(int64_t max_new, int64_t max_context, int64_t window)
{
    int64_t span = max_context;
    if (window && window + max_new + kTile < span)
        span = window + max_new + kTile;
    return (span + kTile - 1) / kTile;
}

// Whether the prompt kernel is the faster one (it takes 128 channels).  Its
// workgroups of 256 rows take 2.3 us for 64 keys, one a CU; the split kernel
// takes about 6 us for 32 rows in each of eight waves a CU, and shares any work
// out evenly.  So up to 32 rows a key head, and where the row blocks leave too
// many CUs idle, the split kernel runs.  Both, us, 32 query heads on 2 key
// heads: one request of 512 tokens behind 8000 235 / 133, of 1024 alone 37 / 55,
// 16 of up to 100 behind up to 3000 85 / 132, eight of up to 1024 67 / 108.
// With 64 channels the split kernel was the faster everywhere from 40 tokens
// to eight prompts of up to 4096 (an eight-wave prompt kernel: 264 / 260 there,
// 47 / 35 for eight of up to 1024).
bool prompt_preferred(int64_t tokens, int64_t requests, int64_t kv_heads, int64_t head_dim, int64_t group, int64_t max_new)
{
    if (max_new * group <= 32 || head_dim != 128)
        return false;
    const double cus = device_cu_count();
    const double rows = (double)tokens * (double)group;
    const double blocks = (rows / 256 + (double)requests) * (double)kv_heads, units = (rows / 32 + (double)requests) * (double)kv_heads;
    return 2.3 * (blocks < cus ? 1.0 : blocks / cus) <= 6.0 * units / (8 * cus);
}

struct SplitShape {
    int rt, units;
    int64_t live; // units of all requests, by the number of tokens
    bool sparse;  // a fraction of requests times units
    int groups;   // workgroups of the streamed form; 0: one a unit
};

// `rows`: the most query rows of a key head.  `ranges`: whether to take ranges
// however many units there are.
SplitShape split_shape(int64_t tokens, int64_t requests, int64_t kv_heads, int64_t head_dim, int64_t rows, int64_t group,
                       int64_t max_new, int64_t max_context, int64_t window, bool ranges)
{
    SplitShape p;
    p.rt = rows <= 16 ? 1 : 2;
    p.units = (int)((rows + 16 * p.rt - 1) / (16 * p.rt) * kv_heads);
    p.live = (tokens * group / (16 * p.rt) + requests) * kv_heads;
    p.sparse = requests * p.units > 2 * p.live && p.live < (1 << 23); // (a grid has fewer than 2^32 threads a side)
    const int64_t tiles = longest_walk(max_new, max_context, window);
    const int64_t gaps = 2 * (1 + kUnitCost) * (tokens * group / (16 * p.rt) + 1) * kv_heads; // tokens of no request
    const int64_t all = (tiles + kUnitCost) * requests * p.units + gaps;
    // What the device's sums can reach (in int32) whatever the lengths it finds:
    // without a causal mask a window bounds no request's keys, if it has more
    // queries than max_new.
    const int64_t most = ((max_context + kTile - 1) / kTile + kUnitCost) * requests * p.units + gaps;
    p.groups = device_cu_count() * split_groups((int)head_dim, p.rt);
    // One workgroup a unit where a unit is short, or where units fill the chip
    // some times over (then the dispatch balances them, also the unequal row
    // blocks of prompts, and nothing has to be joined: 1264 units of up to 66
    // tiles, 16 heads of 64, take 90 us so; in ranges an earlier form took 191,
    // and 30 for the join, where it took 111 so).  With a block of rows a request,
    // not if contexts may be long: a single long one among them would be one
    // workgroup's work (192 tokens behind 1000, 16 heads of 64: 58 us so, 67 in
    // ranges, but 686 and 113 if one of them stands behind 131072; all behind 4000
    // 237 and 244, behind 8000 473 and 481).
    const bool fill = !ranges && requests * p.units >= 4 * (int64_t)p.groups && (p.units > kv_heads || tiles <= 64);
    if (tiles <= 8 || most >= (int64_t(1) << 31) - (1 << 20) || fill)
        p.groups = 0;
    else if (all < kMinRange * (int64_t)p.groups)
        p.groups = (int)((all + kMinRange - 1) / kMinRange);
    return p;
}

// What a call launches.
struct AttnPlan {
    bool prompt;      // the prompt kernel, else the split kernel of shape `main`,
    int main_least;   // for the requests with at least so many rows a key head,
    SplitShape main;
    bool rest;        // and the split kernel of shape `few` for the others
    SplitShape few;
};

AttnPlan attn_plan(int64_t tokens, int64_t requests, int64_t kv_heads, int64_t head_dim, int64_t group, int64_t max_new,
                   int64_t max_context, int64_t window)
{
    AttnPlan p = {};
    p.prompt = prompt_preferred(tokens, requests, kv_heads, head_dim, group, max_new);
    p.main = split_shape(tokens, requests, kv_heads, head_dim, max_new * group, group, max_new, max_context, window, false);
    // The prompt kernel, and the split kernel with a workgroup a unit, give all
    // the keys of a row block to one workgroup.  Where a request may have few rows
    // (some have fewer than max_new tokens) behind more keys than prompts have,
    // those with up to 1024 go to the split kernel in ranges.  Us, before and after,
    // 32 heads on 2: a prompt of 4096 beside one token behind 131072 3336 / 184,
    // beside 8 of them 3316 / 218, beside 64 3333 / 400; one of 2048 beside 63 tokens
    // behind 8000 250 / 113; eight chunks of up to 512 behind 15000, which gain
    // nothing, 582 / 585.
    const int64_t few_new = group < 1024 ? 1024 / group : 1;
    const bool serial = p.prompt || p.main.groups == 0;
    if (serial && max_new > few_new && tokens < requests * max_new &&
        longest_walk(max_new, max_context, window) >= (max_new + kTile - 1) / kTile + long_walk(p.prompt, p.main.sparse)) {
        p.few = split_shape(tokens, requests, kv_heads, head_dim, few_new * group, group, few_new, max_context, window, true);
        p.rest = p.few.groups > 0;
        p.main_least = p.rest ? (int)(few_new * group) + 1 : 0;
    }
    return p;
}

template <int D, int RT, int DT, int LAYOUT, bool ONCE>
hipError_t launch_split(const KvAttnArgs &a, const SplitShape &p, hipStream_t stream)
{
    if (p.groups == 0) {
        const dim3 grid = p.sparse ? dim3((unsigned)p.live) : dim3((unsigned)p.units, (unsigned)a.requests);
        kv_unit_kernel<D, RT, DT, LAYOUT, ONCE><<<grid, dim3(64 * kWaves), 0, stream>>>(a, p.sparse);
        return hipGetLastError();
    }
    const int bound = a.max_new * a.group, rows = bound < a.most_rows ? bound : a.most_rows; // of a key head
    const int most = rows < 16 * RT ? rows : 16 * RT;                                      // of a unit
    // The join that has fewer workgroups.  (By ranges always: 83 us for 79 for two
    // requests of five tokens, 32 heads on 8.)
    const bool by_ranges = (int64_t)rows * a.kv_heads * a.requests > (int64_t)p.groups * most;
    kv_stream_kernel<D, RT, DT, LAYOUT, ONCE><<<dim3((unsigned)p.groups), dim3(64 * kWaves), 0, stream>>>(a, by_ranges);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (by_ranges)
        kv_join_kernel<D, RT, DT, true><<<dim3((unsigned)p.groups, (unsigned)most), dim3(kThreads), 0, stream>>>(a, p.groups);
    else
        kv_join_kernel<D, RT, DT, false><<<dim3((unsigned)rows, (unsigned)a.kv_heads, (unsigned)a.requests), dim3(kThreads), 0, stream>>>(a, p.groups);
    return hipGetLastError();
}

template <int D, int RT, int DT, bool ONCE>
hipError_t launch_layout(const KvAttnArgs &a, const SplitShape &p, hipStream_t stream)
{
    if (a.block_shift < 6)
        return launch_split<D, RT, DT, kNarrow, ONCE>(a, p, stream);
    return a.block_shift == 6 ? launch_split<D, RT, DT, kWhole, ONCE>(a, p, stream)
                              : launch_split<D, RT, DT, kHalf, ONCE>(a, p, stream);
}

template <int D, int DT>
hipError_t launch_dim(const KvAttnArgs &a, const SplitShape &p, hipStream_t stream)
{
    if (p.rt == 1)
        return launch_layout<D, 1, DT, true>(a, p, stream);
    return p.units == a.kv_heads ? launch_layout<D, 2, DT, true>(a, p, stream) : launch_layout<D, 2, DT, false>(a, p, stream);
}

} // namespace

int64_t kv_attention_workspace(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                               int64_t requests, int64_t max_new, int64_t max_context, int64_t window)
{
    const AttnPlan p = attn_plan(tokens, requests, kv_heads, head_dim, q_heads / kv_heads, max_new, max_context, window);
    auto bytes = [&](const SplitShape &f) {
        return (parts_offset(requests, f.groups) + (int64_t)f.groups * 2 * piece_floats((int)head_dim, f.rt)) * (int64_t)sizeof(float);
    };
    if (p.rest)
        return bytes(p.few); // (nothing is left to join by the others)
    return p.prompt || p.main.groups == 0 ? 0 : bytes(p.main);
}

namespace {

hipError_t launch_split_any(const KvAttnArgs &a, const SplitShape &p, int dtype, hipStream_t stream)
{
    if (a.head_dim == 64)
        return dtype == QW_F16 ? launch_dim<64, QW_F16>(a, p, stream) : launch_dim<64, QW_BF16>(a, p, stream);
    if (a.head_dim == 128)
        return dtype == QW_F16 ? launch_dim<128, QW_F16>(a, p, stream) : launch_dim<128, QW_BF16>(a, p, stream);
    return hipErrorInvalidValue;
}

} // namespace

hipError_t launch_kv_attention(const KvAttnArgs &a, int dtype, hipStream_t stream)
{
    const AttnPlan p = attn_plan(a.tokens, a.requests, a.kv_heads, a.head_dim, a.group, a.max_new, a.max_context, a.window);
    KvAttnArgs part = a;
    part.least_rows = p.main_least;
    const hipError_t e = p.prompt ? launch_kv_prompt(part, dtype, stream) : launch_split_any(part, p.main, dtype, stream);
    if (e != hipSuccess || !p.rest)
        return e;
    part.zero_rest = false;
    part.least_rows = 0;
    part.most_rows = p.main_least - 1;
    return launch_split_any(part, p.few, dtype, stream);
}

} // namespace qw
