// kv_cache.hip -- the quantizing write into the paged int8 KV cache, and
// the read back.
//
// Write.  The new tokens of one call that fall into one block form a run
// (consecutive slots).  With o the run's first offset in the block, per head
//
//   S' = fp32(max |x| / 127) over the run (0 below 2^-100)
//   S  = o > 0 ? max(S_old, S') : S'
//   q  = clamp(round_half_even(fp32(x / S)), -127, 127)      (S = 0: 0)
//   q_kept = round_half_even(fp32(q_kept * fp32(S_old / S))) where S > S_old
//
// so a block's scale is the largest value that its live tokens brought, a
// token at offset 0 starts the block afresh, and nothing before the run is
// read unless the scale grows.
//
// Bound by HBM for prompts (2 bytes in, 1 byte out an element) and by
// latency for single tokens.  A wave owns a run (all four waves of the
// workgroup, where the workgroup's window of tokens holds only one): it
// reads the run twice, for the maximum and for the codes; the second read
// comes from L2.  Values are stored transposed: a lane packs 16 tokens of
// two channels into two 16-byte stores.
//
// This unit is compiled without floating-point contraction: codes and
// scales are bit-exact by the formulas above.
#include "kv_device.h"
#include "kv_internal.h"

namespace qw {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t code_of(float x, float s)
{
    const float r = fminf(fmaxf(rintf(x / s), -127.0f), 127.0f);
    return (uint32_t)(int)r & 0xffu;
}

__device__ __forceinline__ uint32_t rescaled(uint32_t byte, float ratio)
{
    return (uint32_t)(int)rintf((float)(int8_t)byte * ratio) & 0xffu;
}

__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float ratio)
{
    return rescaled(w & 0xffu, ratio) | rescaled(w >> 8 & 0xffu, ratio) << 8 | rescaled(w >> 16 & 0xffu, ratio) << 16 |
           rescaled(w >> 24, ratio) << 24;
}

// One run of `len` tokens from token t on, at offset `off` of block `blk`,
// for one head and for keys (VALUES false) or values, by NW waves (this one
// is `wave` of them).
template <int DT, int D, int NW, bool VALUES>
__device__ void write_run(const KvCacheArgs &a, int64_t t, int64_t blk, int off, int len, int head, int wave, float *lds)
{
    constexpr int LPT = D / 8;   // lanes a token of a 16-byte-a-lane read
    constexpr int TPW = 64 / LPT; // tokens a wave reads at once
    const int lane = __lane_id();
    const int64_t block = int64_t(1) << a.block_shift;
    const int64_t stride = VALUES ? a.v_stride : a.k_stride;
    const uint16_t *x = (VALUES ? a.v : a.k) + t * stride + (int64_t)head * D;
    const int64_t bh = blk * a.kv_heads + head;
    int8_t *codes = (VALUES ? a.v_cache : a.k_cache) + bh * block * D;
    float *scale = (VALUES ? a.v_scales : a.k_scales) + bh;

    float top = 0.0f;
    for (int i = wave * TPW + lane / LPT; i < len; i += NW * TPW) {
        float f[8];
        unpack8<DT>(*reinterpret_cast<const u32x4_t *>(x + i * stride + (lane & (LPT - 1)) * 8), f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = fmaxf(top, fabsf(f[e]));
    }
    top = wave_max_f32(top);
    const float was = off > 0 ? *scale : 0.0f;
    if (NW > 1) {
        if (lane == 0)
            lds[wave] = top;
        __syncthreads(); // after it every wave has read `was`
#pragma unroll
        for (int w = 0; w < NW; ++w)
            top = fmaxf(top, lds[w]);
    }
    float s = top / 127.0f;
    s = s < kKvScaleFloor ? 0.0f : s;
    const bool grow = s > was;
    s = grow ? s : was;
    const bool move = off > 0 && grow && was > 0.0f;
    const float ratio = move ? was / s : 1.0f;
    if (wave == 0 && lane == 0)
        *scale = s;

    if (!VALUES) {
        if (move)
            for (int i = (wave * 64 + lane) * 16; i < off * D; i += NW * 64 * 16) {
                u32x4_t *p = reinterpret_cast<u32x4_t *>(codes + i);
                const u32x4_t c = *p;
                *p = (u32x4_t){rescaled4(c.x, ratio), rescaled4(c.y, ratio), rescaled4(c.z, ratio),
                               rescaled4(c.w, ratio)};
            }
        for (int i = wave * TPW + lane / LPT; i < len; i += NW * TPW) {
            const int d = (lane & (LPT - 1)) * 8;
            float f[8];
            unpack8<DT>(*reinterpret_cast<const u32x4_t *>(x + i * stride + d), f);
            u32x2_t c = {0, 0};
            if (s > 0.0f) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    c.x |= code_of(f[e], s) << (8 * e);
                    c.y |= code_of(f[4 + e], s) << (8 * e);
                }
            }
            *reinterpret_cast<u32x2_t *>(codes + (int64_t)(off + i) * D + d) = c;
        }
    } else {
        constexpr int LPS = D / 2;                        // lanes of a 16-token segment: two channels each
        constexpr int SPW = LPS >= 64 ? 1 : 64 / LPS;     // segments a wave writes at once
        constexpr int REP = LPS > 64 ? LPS / 64 : 1;      // channel groups of a wave
        const int d_lane = 2 * (lane & (LPS < 64 ? LPS - 1 : 63));
        const int first = move ? 0 : off / 16, last = (off + len - 1) / 16;
        for (int seg = first + wave * SPW + lane / (LPS < 64 ? LPS : 64); seg <= last; seg += NW * SPW) {
            const int lo = seg * 16;
#pragma unroll
            for (int rep = 0; rep < REP; ++rep) {
                const int d = d_lane + rep * 128;
                int8_t *row0 = codes + (int64_t)d * block + lo, *row1 = row0 + block;
                u32x4_t c0 = {0, 0, 0, 0}, c1 = {0, 0, 0, 0};
                // codes before the run stay (at the new scale); places behind it
                // are not live, and keep what they hold
                if (lo < off || lo + 16 > off + len) {
                    c0 = *reinterpret_cast<const u32x4_t *>(row0);
                    c1 = *reinterpret_cast<const u32x4_t *>(row1);
                    if (move && lo < off) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const int n = off - lo - 4 * v; // codes of this word that lie before the run
                            const uint32_t live = n >= 4 ? ~0u : (n > 0 ? (1u << (8 * n)) - 1 : 0u);
                            c0[v] = (c0[v] & ~live) | (rescaled4(c0[v], ratio) & live);
                            c1[v] = (c1[v] & ~live) | (rescaled4(c1[v], ratio) & live);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int i = lo + j - off;
                    if (i >= 0 && i < len) {
                        const uint32_t pair = *reinterpret_cast<const uint32_t *>(x + i * stride + d);
                        const uint32_t keep = ~(0xffu << (8 * (j & 3)));
                        const uint32_t u = s > 0.0f ? code_of(Act<DT>::lo(pair), s) : 0u;
                        const uint32_t w = s > 0.0f ? code_of(Act<DT>::hi(pair), s) : 0u;
                        c0[j >> 2] = (c0[j >> 2] & keep) | u << (8 * (j & 3));
                        c1[j >> 2] = (c1[j >> 2] & keep) | w << (8 * (j & 3));
                    }
                }
                *reinterpret_cast<u32x4_t *>(row0) = c0;
                *reinterpret_cast<u32x4_t *>(row1) = c1;
            }
        }
    }
}

// Grid: windows of WIN tokens, heads, keys and values.
template <int DT, int D, int WIN>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvCacheArgs a)
{
    __shared__ float lds[kThreads / 64];
    const int lane = __lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.x * WIN;
    const int head = blockIdx.y;
    const int64_t n_slots = a.num_blocks << a.block_shift;
    const int block = 1 << a.block_shift;

    // A run begins where the slot before is not the one below, or at a block's
    // start.  Slots outside the cache (-1: padding) belong to no run.
    const int64_t mine = t0 + lane;
    bool leads = false;
    if (lane < WIN && mine < a.tokens) {
        const int64_t s = a.slots[mine];
        if (s >= 0 && s < n_slots)
            leads = (s & (block - 1)) == 0 || mine == 0 || (int64_t)a.slots[mine - 1] + 1 != s;
    }
    uint64_t leaders = __ballot(leads);
    const bool alone = __popcll(leaders) == 1;
    for (int n = 0; leaders; ++n) {
        const int l = __ffsll((unsigned long long)leaders) - 1;
        leaders &= leaders - 1;
        if (!alone && (n & 3) != wave)
            continue;
        const int64_t t = t0 + l;
        const int64_t slot = a.slots[t];
        const int off = (int)(slot & (block - 1)), most = block - off;
        int len = 0;
        for (int i = 0; i < most; i += 64) {
            const int64_t at = t + i + lane;
            const bool same = i + lane < most && at < a.tokens && (int64_t)a.slots[at] == slot + i + lane;
            const uint64_t b = __ballot(same);
            const int more = ~b ? __ffsll((unsigned long long)~b) - 1 : 64;
            len += more;
            if (more < 64)
                break;
        }
        const int64_t blk = slot >> a.block_shift;
        if (alone) {
            if (blockIdx.z == 0)
                write_run<DT, D, 4, false>(a, t, blk, off, len, head, wave, lds);
            else
                write_run<DT, D, 4, true>(a, t, blk, off, len, head, wave, lds);
        } else {
            if (blockIdx.z == 0)
                write_run<DT, D, 1, false>(a, t, blk, off, len, head, 0, lds);
            else
                write_run<DT, D, 1, true>(a, t, blk, off, len, head, 0, lds);
        }
    }
}

// Read: 64 tokens of one head a workgroup.  Key rows are contiguous; the
// codes of the values go through LDS, read with lanes over tokens (the
// contiguous direction in the cache) and written out with lanes over
// channels.  Rows of slots outside the cache are zero.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvCacheArgs a)
{
    constexpr int LPT = D / 8;
    constexpr int PITCH = D + 4; // bytes: an odd number of banks between tokens
    __shared__ __attribute__((aligned(16))) uint8_t tile[64 * PITCH];
    const int tid = threadIdx.x, lane = __lane_id(), wave = tid >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * 64;
    const int head = blockIdx.y;
    const int64_t n_slots = a.num_blocks << a.block_shift;
    const int64_t block = int64_t(1) << a.block_shift;
    const bool values = blockIdx.z != 0;

    if (values) {
        const int64_t t = t0 + lane;
        const int64_t s = t < a.tokens ? a.slots[t] : -1;
        if (s >= 0 && s < n_slots) {
            const int8_t *p = a.v_cache + ((s >> a.block_shift) * a.kv_heads + head) * block * D + (s & (block - 1));
#pragma unroll 8
            for (int d = wave * (D / 4); d < (wave + 1) * (D / 4); ++d)
                tile[lane * PITCH + d] = (uint8_t)p[d * block];
        }
        __syncthreads();
    }
    for (int i = tid / LPT; i < 64; i += kThreads / LPT) {
        const int64_t t = t0 + i;
        if (t >= a.tokens)
            break;
        const int d = (tid & (LPT - 1)) * 8;
        const int64_t s = a.slots[t];
        u32x2_t c = {0, 0};
        float scale = 0.0f;
        if (s >= 0 && s < n_slots) {
            const int64_t bh = (s >> a.block_shift) * a.kv_heads + head;
            scale = (values ? a.v_scales : a.k_scales)[bh];
            if (values) {
                c.x = *reinterpret_cast<const uint32_t *>(tile + i * PITCH + d);
                c.y = *reinterpret_cast<const uint32_t *>(tile + i * PITCH + d + 4);
            } else {
                c = *reinterpret_cast<const u32x2_t *>(a.k_cache + (bh * block + (s & (block - 1))) * D + d);
            }
        }
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = (float)(int8_t)(c.x >> (8 * e) & 0xffu) * scale;
            f[4 + e] = (float)(int8_t)(c.y >> (8 * e) & 0xffu) * scale;
        }
        uint16_t *out = (values ? a.v + t * a.v_stride : a.k + t * a.k_stride) + (int64_t)head * D + d;
        *reinterpret_cast<u32x4_t *>(out) = pack8<DT>(f);
    }
}

template <int DT, int D>
void write_dim(const KvCacheArgs &a, hipStream_t stream)
{
    // One token a workgroup while that keeps the number of workgroups low
    // (runs are single tokens in decode, and each then has its own workgroup);
    // windows of 16 for prompts, whose runs fill blocks of 16 or more.
    if (a.tokens <= 2048)
        kv_write_kernel<DT, D, 1><<<dim3((unsigned)a.tokens, (unsigned)a.kv_heads, 2), dim3(kThreads), 0, stream>>>(a);
    else
        kv_write_kernel<DT, D, 16><<<dim3((unsigned)((a.tokens + 15) / 16), (unsigned)a.kv_heads, 2), dim3(kThreads), 0, stream>>>(a);
}

template <int DT, int D>
void read_dim(const KvCacheArgs &a, hipStream_t stream)
{
    kv_read_kernel<DT, D><<<dim3((unsigned)((a.tokens + 63) / 64), (unsigned)a.kv_heads, 2), dim3(kThreads), 0, stream>>>(a);
}

} // namespace

hipError_t launch_kv_write(const KvCacheArgs &a, int dtype, hipStream_t stream)
{
    if (a.head_dim == 64)
        dtype == QW_F16 ? write_dim<QW_F16, 64>(a, stream) : write_dim<QW_BF16, 64>(a, stream);
    else if (a.head_dim == 128)
        dtype == QW_F16 ? write_dim<QW_F16, 128>(a, stream) : write_dim<QW_BF16, 128>(a, stream);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCacheArgs &a, int dtype, hipStream_t stream)
{
    if (a.head_dim == 64)
        dtype == QW_F16 ? read_dim<QW_F16, 64>(a, stream) : read_dim<QW_BF16, 64>(a, stream);
    else if (a.head_dim == 128)
        dtype == QW_F16 ? read_dim<QW_F16, 128>(a, stream) : read_dim<QW_BF16, 128>(a, stream);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

} // namespace qw
